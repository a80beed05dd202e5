// Microscaled 4-bit floating point (E2M1 codes with a scale for each block along a GEMM operand's
// contraction axis): the formats' scales and codes, and where a block's scale lies.
//
// E2M1 has the values 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives, two codes a byte (the even
// element in the low half). Codes are rounded to nearest, ties to the even code, saturating.
//   MX: blocks of 32; scale 2^(floor(log2 amax) - 2), stored as its exponent + 127 (E8M0). The
//       exponent comes from amax's bits and x / scale is exact, so nothing is rounded but the
//       code. A block with an infinity or NaN gets the scale 0xff (NaN).
//   NV: blocks of 16; scale s = E4M3(RN(RN(amax / g) / 6)) under a power of two g for each row, the
//       smallest with rowmax / g <= 6 * 448, so that the row's largest block has a scale of 224
//       to 448. RN(x / g / s) is decided against E2M1's midpoints as the exact quotient is: a
//       midpoint (at most 3 significant bits: 1.75, 3.5) times s (4) has at most 7 significant bits
//       and x has 8, so where x / g is not that product it is at least 2^-8 of it away, and fp32
//       rounds by 2^-24. A row with an infinity or NaN gets g = NaN. Blocks whose scale rounds
//       to 0 have codes of 0.
//
// Scale tiles: the scales of 128 rows x 4 consecutive blocks are 512 bytes together, in the order
// in which tcgen05.cp puts them into tensor memory (a row's four bytes side by side).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "fp8.cuh"

namespace moe {

template <bool NV>
struct Fp4 {
    static constexpr int BLOCK = NV ? 16 : 32;
    static constexpr int TILE_K = 4 * BLOCK;  // elements along K that one scale tile spans
};

// Byte offset of the four scales of row r in K tile kt (of ktiles).
__host__ __device__ __forceinline__ int64_t fp4_scale_word(int64_t r, int64_t kt, int64_t ktiles) {
    return ((r >> 7) * ktiles + kt) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// Larger magnitude of each half of two bf16 pairs, on their bits: magnitudes order as integers do,
// infinities above numbers and NaN above those.
__device__ __forceinline__ uint32_t absmax2(uint32_t m, uint32_t w) {
    return __vmaxu2(m, w & 0x7fff7fffu);
}
__device__ __forceinline__ uint32_t absmax8(uint32_t m, const uint4 v) {
    return absmax2(absmax2(absmax2(absmax2(m, v.x), v.y), v.z), v.w);
}
__device__ __forceinline__ uint32_t halves_max(uint32_t m) { return max(m & 0xffffu, m >> 16); }

// Eight numbers to eight codes.
__device__ __forceinline__ uint32_t fp4_codes8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// MX scale of a block whose largest magnitude has the bf16 bits `amax`.
struct MxScale {
    uint32_t byte;
    float inv;  // 1 / scale, a power of two
    __device__ __forceinline__ explicit MxScale(uint32_t amax) {
        const int e = (int)(amax >> 7);
        byte = e == 255 ? 255u : (uint32_t)max(e - 2, 0);
        inv = __uint_as_float(e == 255 ? 0x3f800000u : (254u - byte) << 23);
    }
    __device__ __forceinline__ float quot(float x) const { return x * inv; }
    __device__ __forceinline__ uint32_t finish(uint32_t codes) const { return codes; }
    __device__ __forceinline__ uint32_t codes(const uint4 w) const {
        const float v[8] = {bf16_lo(w.x) * inv, bf16_hi(w.x) * inv, bf16_lo(w.y) * inv,
                            bf16_hi(w.y) * inv, bf16_lo(w.z) * inv, bf16_hi(w.z) * inv,
                            bf16_lo(w.w) * inv, bf16_hi(w.w) * inv};
        return fp4_codes8(v);
    }
};

// The code bytes and the scale byte of an MX block given as 16 packed bf16 pairs.
__device__ __forceinline__ uint32_t mx_block(const uint32_t (&w)[16], uint4& codes) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) m = absmax2(m, w[j]);
    const MxScale sc(halves_max(m));
    codes = make_uint4(sc.codes(make_uint4(w[0], w[1], w[2], w[3])),
                       sc.codes(make_uint4(w[4], w[5], w[6], w[7])),
                       sc.codes(make_uint4(w[8], w[9], w[10], w[11])),
                       sc.codes(make_uint4(w[12], w[13], w[14], w[15])));
    return sc.byte;
}

// The power of two of an NV row whose largest magnitude has the bf16 bits `top`: 2688 is
// 1.3125 * 2^11, and bf16's seven fraction bits of 1.3125 are 40.
struct NvRow {
    float g, inv;
    __device__ __forceinline__ explicit NvRow(uint32_t top) {
        const int e = (int)(top >> 7);
        const int q = max(e - 127 - 11 + ((top & 127u) > 40u ? 1 : 0), -126);
        g = __uint_as_float((uint32_t)(q + 127) << 23);
        inv = __uint_as_float((uint32_t)(127 - q) << 23);
        if (top == 0) g = inv = 1.0f;
        if (e == 255) g = __uint_as_float(0x7fffffffu);
    }
};

struct NvScale {
    uint32_t byte;
    float rinv;   // of the row
    float s, rs;  // the scale and its rounded reciprocal; rs is 0 for a scale of 0
    __device__ __forceinline__ NvScale(uint32_t amax, const NvRow& row) {
        const float am = __uint_as_float(amax << 16) * row.inv;
        // RN(am / 6) by the rounded reciprocal and one correction (Markstein), as quot below
        const float sixth = 1.0f / 6.0f, q0 = __fmul_rn(am, sixth);
        const float q = __fmaf_rn(__fmaf_rn(-q0, 6.0f, am), sixth, q0);
        byte = __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
        s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
        rs = s > 0.f ? __frcp_rn(s) : 0.f;
        rinv = row.inv;
    }
    // RN(x / g / s), without a division: as Fp8Scale::quot, with the remainder taken the other way
    // round so that a zero keeps its sign
    __device__ __forceinline__ float quot(float x) const {
        const float y = x * rinv;
        const float q0 = __fmul_rn(y, rs);
        return __fmaf_rn(-__fmaf_rn(q0, s, -y), rs, q0);
    }
    __device__ __forceinline__ uint32_t codes(const uint4 w) const {
        const float v[8] = {quot(bf16_lo(w.x)), quot(bf16_hi(w.x)), quot(bf16_lo(w.y)),
                            quot(bf16_hi(w.y)), quot(bf16_lo(w.z)), quot(bf16_hi(w.z)),
                            quot(bf16_lo(w.w)), quot(bf16_hi(w.w))};
        return finish(fp4_codes8(v));
    }
    __device__ __forceinline__ uint32_t finish(uint32_t codes) const {
        return s > 0.f ? codes : 0u;  // no sign either under a scale of 0
    }
};

// Rows [0, min(rows, *limit)) of X, or of [X | X1], to codes and scales; see fp4.cu.
int launch_quantize_rows_fp4(const __nv_bfloat16* X, const __nv_bfloat16* X1, const int64_t* limit,
                             int64_t rows, int cols, int fmt, uint8_t* Q, uint8_t* S, float* g,
                             cudaStream_t st);

}  // namespace moe
