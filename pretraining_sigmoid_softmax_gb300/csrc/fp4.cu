// Quantisation to microscaled 4-bit floating point and back, and the dispatch of quantised rows
// (the formats: fp4.cuh). All four are bound by memory.
#include <cuda_fp4.h>
#include <cuda_runtime.h>

#include "fp4.cuh"
#include "sizes.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Rows. A thread takes 16 consecutive elements (32 bytes) at a time and keeps up to NIT such
// pieces in registers, so that a row is read once although its largest value (NV) is needed
// first. WPR warps share a row. Blocks of 16 lie in one thread, blocks of 32 in two; the four
// scales of a tile's row are put together by shuffles and stored as one word.
template <bool NV, int WPR, int NIT>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(
    const __nv_bfloat16* __restrict__ X, const __nv_bfloat16* __restrict__ X1,
    const int64_t* __restrict__ limit, int64_t rows, int cols, uint8_t* __restrict__ Q,
    uint8_t* __restrict__ S, float* __restrict__ G) {
    constexpr int ROWS = kThreads / 32 / WPR;  // rows a CTA takes at a time
    __shared__ uint32_t part[NV && WPR > 1 ? kThreads / 32 : 1];
    const int lane = threadIdx.x % 32;
    const int t = threadIdx.x % (32 * WPR);
    const int np0 = cols / 16;                 // pieces of X's row
    const int np = X1 ? 2 * np0 : np0;
    const int64_t ktiles = np * 16 / Fp4<NV>::TILE_K;
    int64_t n = rows;
    if (limit) n = min(n, *limit);
    for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < n; r0 += (int64_t)gridDim.x * ROWS) {
        const int64_t r = r0 + threadIdx.x / (32 * WPR);
        const bool in_row = r < n;
        uint4 v[NIT][2];
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            const int p = t + i * 32 * WPR;
            v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
            if (in_row && p < np) {
                const __nv_bfloat16* src = p < np0 ? X + r * cols + 16 * p
                                                   : X1 + r * cols + 16 * (p - np0);
                v[i][0] = reinterpret_cast<const uint4*>(src)[0];
                v[i][1] = reinterpret_cast<const uint4*>(src)[1];
            }
        }
        uint32_t am[NIT];
#pragma unroll
        for (int i = 0; i < NIT; ++i) am[i] = halves_max(absmax8(absmax8(0u, v[i][0]), v[i][1]));
        uint32_t top = 0;
        if constexpr (NV) {
#pragma unroll
            for (int i = 0; i < NIT; ++i) top = max(top, am[i]);
            top = __reduce_max_sync(0xffffffffu, top);
            if constexpr (WPR > 1) {
                if (lane == 0) part[threadIdx.x / 32] = top;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < WPR; ++w) top = max(top, part[threadIdx.x / (32 * WPR) * WPR + w]);
                __syncthreads();
            }
        }
        const NvRow row(top);
        if (NV && in_row && t == 0) G[r] = row.g;
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            const int p = t + i * 32 * WPR;
            if (i * 32 * WPR >= np) break;  // the same for the whole CTA
            uint2 code;
            uint32_t word;
            if constexpr (NV) {
                const NvScale sc(am[i], row);
                code = make_uint2(sc.codes(v[i][0]), sc.codes(v[i][1]));
                word = sc.byte << (8 * (lane & 3));
                word |= __shfl_xor_sync(0xffffffffu, word, 1);
                word |= __shfl_xor_sync(0xffffffffu, word, 2);
            } else {
                const MxScale sc(max(am[i], __shfl_xor_sync(0xffffffffu, am[i], 1)));
                code = make_uint2(sc.codes(v[i][0]), sc.codes(v[i][1]));
                word = sc.byte << (8 * ((lane >> 1) & 3));
                word |= __shfl_xor_sync(0xffffffffu, word, 2);
                word |= __shfl_xor_sync(0xffffffffu, word, 4);
            }
            if (in_row && p < np) {  // np is a multiple of 8: whole tiles of scales
                reinterpret_cast<uint2*>(Q + r * (np * 8))[p] = code;
                constexpr int PT = Fp4<NV>::TILE_K / 16;  // pieces of a tile
                if (lane % PT == 0)
                    *reinterpret_cast<uint32_t*>(S + fp4_scale_word(r, p / PT, ktiles)) = word;
            }
        }
    }
}

// The numbers that codes stand for: E2M1 * scale (* g), one rounding to bf16, which is exact (the
// product has at most 6 significant bits) unless it leaves bf16's range.
template <bool NV>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(
    const uint8_t* __restrict__ Q, const uint8_t* __restrict__ S, const float* __restrict__ G,
    const int64_t* __restrict__ limit, int64_t rows, int cols, __nv_bfloat16* __restrict__ out) {
    const int np = cols / 16;
    const int64_t ktiles = cols / Fp4<NV>::TILE_K;
    constexpr int PT = Fp4<NV>::TILE_K / 16;
    int64_t n = rows;
    if (limit) n = min(n, *limit);
    const int64_t total = n * np;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * kThreads) {
        const int64_t r = i / np;
        const int p = (int)(i - r * np);
        const uint2 code = reinterpret_cast<const uint2*>(Q)[i];
        const uint32_t byte = S[fp4_scale_word(r, p / PT, ktiles) + p % PT / (PT / 4)];
        float s;
        if constexpr (NV)
            s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3))) * G[r];
        else
            s = byte == 255 ? __uint_as_float(0x7fffffffu)
                            : byte ? __uint_as_float(byte << 23) : __uint_as_float(1u << 22);
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = ((j < 4 ? code.x : code.y) >> (8 * (j & 3))) & 0xffu;
            const __half2 h(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)b, __NV_E2M1));
            const float2 f = __half22float2(h);
            w[j] = pack_bf16x2(f.x * s, f.y * s);
        }
        uint4* dst = reinterpret_cast<uint4*>(out) + 2 * i;
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// ------------------------------------------------ columnwise scales, transposed codes
// X is E matrices of K x N bf16, or, with X1, the K = 2 K0 stack of X0 over X1. Column n's codes
// are written as row e N + n of the operand, K-major, its blocks along K.

// NV: largest magnitude of each column (as bits, which order as the magnitudes do; `top` starts at
// zero): a thread takes 8 columns and kTopRows rows.
constexpr int kTopThreads = 128;
constexpr int kTopRows = 128;

__global__ void __launch_bounds__(kTopThreads) column_top_kernel(const __nv_bfloat16* __restrict__ X0,
                                                                 const __nv_bfloat16* __restrict__ X1,
                                                                 int K0, int N,
                                                                 uint32_t* __restrict__ top) {
    const int e = blockIdx.y;
    const int K = X1 ? 2 * K0 : K0;
    const int c = (blockIdx.x * kTopThreads + threadIdx.x) * 8;
    if (c >= N) return;
    const int r0 = blockIdx.z * kTopRows, r1 = min(K, r0 + kTopRows);
    uint4 m = make_uint4(0, 0, 0, 0);
#pragma unroll 8
    for (int r = r0; r < r1; ++r) {
        const __nv_bfloat16* src = r < K0 ? X0 + ((int64_t)e * K0 + r) * N
                                          : X1 + ((int64_t)e * K0 + (r - K0)) * N;
        const uint4 v = *reinterpret_cast<const uint4*>(src + c);
        m = make_uint4(absmax2(m.x, v.x), absmax2(m.y, v.y), absmax2(m.z, v.z), absmax2(m.w, v.w));
    }
    uint32_t* dst = top + (int64_t)e * N + c;
    const uint32_t w[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        atomicMax(dst + 2 * q, w[q] & 0xffffu);
        atomicMax(dst + 2 * q + 1, w[q] >> 16);
    }
}

// Column maxima (bits) to the rows' powers of two, in place.
__global__ void column_g_kernel(float* __restrict__ G, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) G[i] = NvRow(__float_as_uint(G[i])).g;
}

// Tiles of 128 K-rows x 64 columns through shared memory. A thread makes the codes of 32 K
// elements of one column: 16 bytes, one block of 32 or two of 16.
constexpr int kColK = 128;
constexpr int kColN = 64;

template <bool NV>
__global__ void __launch_bounds__(kThreads) quantize_cols_kernel(
    const __nv_bfloat16* __restrict__ X0, const __nv_bfloat16* __restrict__ X1, int K0, int N,
    uint8_t* __restrict__ Qt, uint8_t* __restrict__ S, const float* __restrict__ G) {
    __shared__ __align__(16) uint16_t tile[kColK][kColN + 2];
    __shared__ __align__(16) uint8_t scale[kColN][8];
    const int e = blockIdx.z, n0 = blockIdx.x * kColN, k0 = blockIdx.y * kColK;
    const int K = X1 ? 2 * K0 : K0;  // K0 % 128 == 0: a tile lies in one of the two
    const __nv_bfloat16* src = (k0 < K0 ? X0 + ((int64_t)e * K0 + k0) * N
                                        : X1 + ((int64_t)e * K0 + (k0 - K0)) * N) + n0;
    for (int i = threadIdx.x; i < kColK * (kColN / 8); i += kThreads) {
        const int r = i / (kColN / 8), c8 = i % (kColN / 8);
        const uint4 v = *reinterpret_cast<const uint4*>(src + (int64_t)r * N + 8 * c8);
        uint32_t* dst = reinterpret_cast<uint32_t*>(&tile[r][8 * c8]);
        dst[0] = v.x;
        dst[1] = v.y;
        dst[2] = v.z;
        dst[3] = v.w;
    }
    __syncthreads();
    {
        const int n = threadIdx.x % kColN, q = threadIdx.x / kColN;
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int k = 32 * q + 8 * j + 2 * h;
                w[h] = tile[k][n] | ((uint32_t)tile[k + 1][n] << 16);
            }
            v[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        const uint32_t a = halves_max(absmax8(absmax8(0u, v[0]), v[1]));
        const uint32_t b = halves_max(absmax8(absmax8(0u, v[2]), v[3]));
        const int64_t r = (int64_t)e * N + n0 + n;
        uint4 code;
        if constexpr (NV) {
            NvRow row(0);
            row.g = G[r];
            row.inv = 1.0f / row.g;  // of a power of two: exact
            const NvScale sa(a, row), sb(b, row);
            code = make_uint4(sa.codes(v[0]), sa.codes(v[1]), sb.codes(v[2]), sb.codes(v[3]));
            scale[n][2 * q] = (uint8_t)sa.byte;
            scale[n][2 * q + 1] = (uint8_t)sb.byte;
        } else {
            const MxScale sc(max(a, b));
            code = make_uint4(sc.codes(v[0]), sc.codes(v[1]), sc.codes(v[2]), sc.codes(v[3]));
            scale[n][q] = (uint8_t)sc.byte;
        }
        *reinterpret_cast<uint4*>(Qt + r * (K / 2) + k0 / 2 + 16 * q) = code;
    }
    __syncthreads();
    constexpr int WORDS = kColK / Fp4<NV>::TILE_K;  // scale tiles that a tile's columns pass
    if (threadIdx.x < kColN * WORDS) {
        const int n = threadIdx.x % kColN, w = threadIdx.x / kColN;
        *reinterpret_cast<uint32_t*>(
            S + fp4_scale_word((int64_t)e * N + n0 + n, k0 / Fp4<NV>::TILE_K + w, K / Fp4<NV>::TILE_K)) =
            *reinterpret_cast<const uint32_t*>(&scale[n][4 * w]);
    }
}

// ---------------------------------------------------------- dispatch of quantised rows
// Codes and scales of a row depend on that row alone, so those of an expert-major row are its
// token's: a warp copies a token's codes and scale words to its k rows.
constexpr int kGatherWarps = 8;

__global__ void __launch_bounds__(kGatherWarps * 32) permute_kernel(
    const uint8_t* __restrict__ xq, const uint8_t* __restrict__ sx, const float* __restrict__ gx,
    const int32_t* __restrict__ slot_to_row, int64_t T, int d, int k, int ktiles,
    uint8_t* __restrict__ Xq, uint8_t* __restrict__ sX, float* __restrict__ gX) {
    const int lane = threadIdx.x % 32;
    const int64_t t = (int64_t)blockIdx.x * kGatherWarps + threadIdx.x / 32;
    if (t >= T) return;
    int32_t my_row = -1;
    if (lane < k) my_row = slot_to_row[t * k + lane];
    if (gx && my_row >= 0) gX[my_row] = gx[t];
    const uint4* src = reinterpret_cast<const uint4*>(xq + t * (d / 2));
    const int nvec = d / 32;
    for (int c0 = 0; c0 < nvec; c0 += 32) {  // warp-uniform trip count
        const int c = c0 + lane;
        const bool in = c < nvec;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (in) v = src[c];
        for (int i = 0; i < k; ++i) {
            const int32_t row = __shfl_sync(0xffffffffu, my_row, i);
            if (in && row >= 0) reinterpret_cast<uint4*>(Xq + (int64_t)row * (d / 2))[c] = v;
        }
    }
    for (int c0 = 0; c0 < ktiles; c0 += 32) {
        const int c = c0 + lane;
        const bool in = c < ktiles;
        uint32_t w = 0;
        if (in) w = *reinterpret_cast<const uint32_t*>(sx + fp4_scale_word(t, c, ktiles));
        for (int i = 0; i < k; ++i) {
            const int32_t row = __shfl_sync(0xffffffffu, my_row, i);
            if (in && row >= 0)
                *reinterpret_cast<uint32_t*>(sX + fp4_scale_word(row, c, ktiles)) = w;
        }
    }
}

// Padding rows of each segment (the trailing rows with perm_token < 0; at most MOE_ROW_ALIGN - 1
// per expert): zero codes, scales of zero bits and g = 1, as quantising a zero row gives.
constexpr int kPadSplit = 16;

__global__ void __launch_bounds__(kThreads) pad_rows_kernel(const int64_t* __restrict__ row_offsets,
                                                            const int32_t* __restrict__ perm_token,
                                                            int d, int ktiles,
                                                            uint8_t* __restrict__ Xq,
                                                            uint8_t* __restrict__ sX,
                                                            float* __restrict__ gX) {
    const int e = blockIdx.x;
    const int64_t hi = row_offsets[e + 1];
    int64_t lo = row_offsets[e];
    if (hi - lo > MOE_ROW_ALIGN - 1) lo = hi - (MOE_ROW_ALIGN - 1);
    const int per_row = d / 32;
    for (int64_t i = (int64_t)blockIdx.y * kThreads + threadIdx.x; i < (hi - lo) * per_row;
         i += (int64_t)gridDim.y * kThreads) {
        const int64_t r = lo + i / per_row;
        const int c = (int)(i % per_row);
        if (perm_token[r] >= 0) continue;
        reinterpret_cast<uint4*>(Xq + r * (d / 2))[c] = make_uint4(0, 0, 0, 0);
        if (c < ktiles) *reinterpret_cast<uint32_t*>(sX + fp4_scale_word(r, c, ktiles)) = 0;
        if (gX && c == 0) gX[r] = 1.0f;
    }
}

template <bool NV, int WPR, int NIT>
int launch_rows(const __nv_bfloat16* X, const __nv_bfloat16* X1, const int64_t* limit, int64_t rows,
                int cols, uint8_t* Q, uint8_t* S, float* g, cudaStream_t st) {
    int64_t blocks = cdiv(rows, kThreads / 32 / WPR);
    const int64_t cap = (int64_t)sm_count() * 16;
    if (blocks > cap) blocks = cap;
    quantize_rows_kernel<NV, WPR, NIT><<<(unsigned)blocks, kThreads, 0, st>>>(X, X1, limit, rows, cols,
                                                                             Q, S, g);
    return launch_status();
}

template <bool NV>
int rows_by_width(const __nv_bfloat16* X, const __nv_bfloat16* X1, const int64_t* limit, int64_t rows,
                  int cols, uint8_t* Q, uint8_t* S, float* g, cudaStream_t st) {
    const int width = X1 ? 2 * cols : cols;
    // A warp holds rows of up to 4096 elements; wider ones, and rows too few to fill the GPU with
    // a warp each, take a CTA of eight.
    if (width > 4096 || rows < 8 * (int64_t)sm_count()) {
        if (width <= 4096) return launch_rows<NV, 8, 1>(X, X1, limit, rows, cols, Q, S, g, st);
        if (width <= 8192) return launch_rows<NV, 8, 2>(X, X1, limit, rows, cols, Q, S, g, st);
        return launch_rows<NV, 8, 8>(X, X1, limit, rows, cols, Q, S, g, st);
    }
    if (width <= 1024) return launch_rows<NV, 1, 2>(X, X1, limit, rows, cols, Q, S, g, st);
    if (width <= 2048) return launch_rows<NV, 1, 4>(X, X1, limit, rows, cols, Q, S, g, st);
    return launch_rows<NV, 1, 8>(X, X1, limit, rows, cols, Q, S, g, st);
}

bool fmt_ok(int fmt) { return fmt == MOE_FP4_MX || fmt == MOE_FP4_NV; }
// NV has a power of two for each row, MX has none.
bool g_ok(int fmt, const float* g) { return (fmt == MOE_FP4_NV) == (g != nullptr); }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

int launch_quantize_rows_fp4(const __nv_bfloat16* X, const __nv_bfloat16* X1, const int64_t* limit,
                             int64_t rows, int cols, int fmt, uint8_t* Q, uint8_t* S, float* g,
                             cudaStream_t st) {
    return fmt == MOE_FP4_NV ? rows_by_width<true>(X, X1, limit, rows, cols, Q, S, g, st)
                             : rows_by_width<false>(X, X1, limit, rows, cols, Q, S, g, st);
}

}  // namespace moe

using namespace moe;

extern "C" int64_t moe_fp4_scale_bytes(int64_t rows, int cols, int fmt) {
    if (rows <= 0 || cols <= 0 || cols % 128 != 0 || !fmt_ok(fmt)) return 0;
    return cdiv(rows, 128) * 128 * (cols / (fmt == MOE_FP4_NV ? 16 : 32));
}

extern "C" int moe_quantize_rows_fp4(const moe_bf16* X, const moe_bf16* X1, const int64_t* rows_limit,
                                     int64_t rows, int cols, int fmt, uint8_t* Q, uint8_t* S, float* g,
                                     moe_stream_t stream) {
    if (!X || !Q || !S || !fmt_ok(fmt) || !g_ok(fmt, g)) return MOE_ERR_INVALID_ARG;
    if (rows <= 0 || cols <= 0) return MOE_ERR_INVALID_ARG;
    if (cols % 128 != 0 || (X1 ? 2 * (int64_t)cols : cols) > kFp4MaxCols) return MOE_ERR_UNSUPPORTED;
    if (!aligned16(X) || (X1 && !aligned16(X1)) || !aligned16(Q) || !aligned16(S) || !aligned4(g))
        return MOE_ERR_INVALID_ARG;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    return launch_quantize_rows_fp4(reinterpret_cast<const __nv_bfloat16*>(X),
                                    reinterpret_cast<const __nv_bfloat16*>(X1), rows_limit, rows, cols,
                                    fmt, Q, S, g, (cudaStream_t)stream);
}

extern "C" int moe_quantize_cols_fp4(const moe_bf16* X0, const moe_bf16* X1, int E, int K0, int N,
                                     int fmt, uint8_t* Qt, uint8_t* S, float* g, moe_stream_t stream) {
    if (!X0 || !Qt || !S || !fmt_ok(fmt) || !g_ok(fmt, g)) return MOE_ERR_INVALID_ARG;
    if (E <= 0 || K0 <= 0 || N <= 0) return MOE_ERR_INVALID_ARG;
    if (K0 % 128 != 0 || N % 128 != 0 || K0 > kFp4MaxCols || N > kFp4MaxCols || E > 65535)
        return MOE_ERR_UNSUPPORTED;
    if (!aligned16(X0) || (X1 && !aligned16(X1)) || !aligned16(Qt) || !aligned16(S) || !aligned4(g))
        return MOE_ERR_INVALID_ARG;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    cudaStream_t st = (cudaStream_t)stream;
    const auto* x0 = reinterpret_cast<const __nv_bfloat16*>(X0);
    const auto* x1 = reinterpret_cast<const __nv_bfloat16*>(X1);
    const int K = X1 ? 2 * K0 : K0;
    const dim3 grid((unsigned)(N / kColN), (unsigned)(K / kColK), (unsigned)E);
    if (fmt == MOE_FP4_MX) {
        quantize_cols_kernel<false><<<grid, kThreads, 0, st>>>(x0, x1, K0, N, Qt, S, nullptr);
        return launch_status();
    }
    const int64_t n = (int64_t)E * N;
    if (cudaMemsetAsync(g, 0, sizeof(float) * n, st) != cudaSuccess) return MOE_ERR_LAUNCH;
    column_top_kernel<<<dim3((unsigned)cdiv(N, 8 * kTopThreads), (unsigned)E, (unsigned)cdiv(K, kTopRows)),
                        kTopThreads, 0, st>>>(x0, x1, K0, N, reinterpret_cast<uint32_t*>(g));
    column_g_kernel<<<(unsigned)cdiv(n, 256), 256, 0, st>>>(g, n);
    quantize_cols_kernel<true><<<grid, kThreads, 0, st>>>(x0, x1, K0, N, Qt, S, g);
    return launch_status();
}

extern "C" int moe_dequantize_fp4(const uint8_t* Q, const uint8_t* S, const float* g,
                                  const int64_t* rows_limit, int64_t rows, int cols, int fmt,
                                  moe_bf16* out, moe_stream_t stream) {
    if (!Q || !S || !out || !fmt_ok(fmt) || !g_ok(fmt, g)) return MOE_ERR_INVALID_ARG;
    if (rows <= 0 || cols <= 0) return MOE_ERR_INVALID_ARG;
    if (cols % 128 != 0) return MOE_ERR_UNSUPPORTED;
    if (!aligned16(Q) || !aligned16(S) || !aligned16(out) || !aligned4(g)) return MOE_ERR_INVALID_ARG;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    int64_t blocks = cdiv(rows * (cols / 16), kThreads);
    const int64_t cap = (int64_t)sm_count() * 32;
    if (blocks > cap) blocks = cap;
    auto* o = reinterpret_cast<__nv_bfloat16*>(out);
    if (fmt == MOE_FP4_NV)
        dequantize_kernel<true><<<(unsigned)blocks, kThreads, 0, (cudaStream_t)stream>>>(
            Q, S, g, rows_limit, rows, cols, o);
    else
        dequantize_kernel<false><<<(unsigned)blocks, kThreads, 0, (cudaStream_t)stream>>>(
            Q, S, g, rows_limit, rows, cols, o);
    return launch_status();
}

extern "C" int moe_permute_fp4(const uint8_t* xq, const uint8_t* sx, const float* gx,
                               const int32_t* slot_to_row, const int32_t* perm_token,
                               const int64_t* row_offsets, int64_t T, int d, int E, int k, int fmt,
                               uint8_t* Xq, uint8_t* sX, float* gX, moe_stream_t stream) {
    if (!xq || !sx || !slot_to_row || !perm_token || !row_offsets || !Xq || !sX || !fmt_ok(fmt) ||
        !g_ok(fmt, gx) || !g_ok(fmt, gX))
        return MOE_ERR_INVALID_ARG;
    if (T <= 0 || d <= 0 || E <= 0 || k <= 0) return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts || k > E || k > 32 || d % 128 != 0) return MOE_ERR_UNSUPPORTED;
    if (!aligned16(xq) || !aligned16(sx) || !aligned16(Xq) || !aligned16(sX) || !aligned4(gx) ||
        !aligned4(gX))
        return MOE_ERR_INVALID_ARG;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    cudaStream_t st = (cudaStream_t)stream;
    const int ktiles = d / (fmt == MOE_FP4_NV ? Fp4<true>::TILE_K : Fp4<false>::TILE_K);
    permute_kernel<<<(unsigned)cdiv(T, kGatherWarps), kGatherWarps * 32, 0, st>>>(
        xq, sx, gx, slot_to_row, T, d, k, ktiles, Xq, sX, gX);
    pad_rows_kernel<<<dim3(E, kPadSplit), kThreads, 0, st>>>(row_offsets, perm_token, d, ktiles, Xq, sX,
                                                            gX);
    return launch_status();
}
