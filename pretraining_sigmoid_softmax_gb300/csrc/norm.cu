// Residual addition and root-mean-square norm in front of the MoE layer, and its backward.
//
// Forward, per token: z = residual + x (rounded to the residual stream's type), rstd =
// 1 / sqrt(mean(z^2) + eps), y = z rstd w; y leaves as bf16 and, for the FP8 experts, as E4M3
// codes under one scale per row (amax / 448 of the unrounded y, 1 for a zero row).
// Backward, with xhat = z rstd and g = dy w: dz = rstd (g - xhat mean(g xhat)) + dres,
// dw = sum over tokens of dy xhat.
//
// Both are bound by HBM: every tensor is read or written once. A row stays in registers (forward)
// or shared memory (backward) between its loads and its stores, and the sum of squares and the
// row's largest value come from one pass. Times below are of launches in a graph, fractions of
// the rate at which a plain copy moves the same bytes (6.78 TB/s).
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "common.cuh"
#include "sizes.h"

namespace moe {
namespace {

// Eight consecutive values of a row as floats.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[2 * q] = bf16_lo(w[q]);
        v[2 * q + 1] = bf16_hi(w[q]);
    }
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// fp32 streams in one 32-byte access each: two 16-byte ones would touch every sector twice.
__device__ __forceinline__ void load8_stream(const float* p, float (&v)[8]) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
                   "=f"(v[7])
                 : "l"(p));
}
__device__ __forceinline__ void load8_stream(const __nv_bfloat16* p, float (&v)[8]) { load8(p, v); }
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
                 "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

// The library's own sums (shared or global memory, 16-byte aligned).
__device__ __forceinline__ void put8(float* p, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// A value as the residual stream stores it.
__device__ __forceinline__ float stored(float v, const __nv_bfloat16*) {
    return __bfloat162float(__float2bfloat16_rn(v));
}
__device__ __forceinline__ float stored(float v, const float*) { return v; }

// Reduces a sum and a maximum over all threads of a row at once, in a fixed order: a butterfly
// within each warp, then (rows of several warps) the warps' values from shared memory in their
// order, behind one barrier. `red` holds a slot per warp and is written once per barrier.
__device__ __forceinline__ void row_reduce(float& s, float& m, float2* red, int nwarps) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if (nwarps == 1) return;  // rows of one warp: no barrier
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = make_float2(s, m);
    __syncthreads();
    s = red[0].x;
    m = red[0].y;
    for (int i = 1; i < nwarps; ++i) {
        s += red[i].x;
        m = fmaxf(m, red[i].y);
    }
}

__device__ __forceinline__ float row_reduce(float s, float2* red, int nwarps) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (nwarps == 1) return s;
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32].x = s;
    __syncthreads();
    s = red[0].x;
    for (int i = 1; i < nwarps; ++i) s += red[i].x;
    return s;
}

// E4M3 codes of four values each in two words, round to nearest even, saturating.
__device__ __forceinline__ uint2 codes8_of(const float (&q)[8]) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const __nv_fp8x2_storage_t a =
            __nv_cvt_float2_to_fp8x2(make_float2(q[4 * h], q[4 * h + 1]), __NV_SATFINITE, __NV_E4M3);
        const __nv_fp8x2_storage_t b =
            __nv_cvt_float2_to_fp8x2(make_float2(q[4 * h + 2], q[4 * h + 3]), __NV_SATFINITE, __NV_E4M3);
        w[h] = (uint32_t)a | ((uint32_t)b << 16);
    }
    return make_uint2(w[0], w[1]);
}

// blockDim = (threads per row, rows per CTA); rows of one warp may share a CTA. Thread i of a
// row owns its vectors i, i + blockDim.x, ... (eight values each), VPT of them at most.
//
// y = (z w) rstd, so the largest |y| is rstd times the largest |z w|, which is known together with
// the sum of squares: one reduction, one barrier. In the quotient of the codes rstd cancels:
// y / sy = z w (448 / max |z w|), a product with one factor per row.
//
// 65,536 x 4096 with an fp32 stream and codes (3.49 GB): 496 us, 1.04 of a copy; with a bf16 stream
// and codes 368 us, 0.97; 8191 x 1024 bf16 (67 MB): 13.6 us, 0.73, of which 2.4 us are those of
// a launch with one row.
template <typename R, int VPT, bool CODES>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(
    const __nv_bfloat16* x, const R* res, const float* __restrict__ w, float eps, int64_t T, int d,
    R* z_out, __nv_bfloat16* y, uint8_t* __restrict__ yq, float* __restrict__ sy,
    float* __restrict__ rstd_out) {
    __shared__ float2 red[32];
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= T) return;  // a whole row (a warp of its own where rows share a CTA)
    const int nvec = d / 8, nwarps = blockDim.x / 32;
    float z[VPT][8];
    float ss = 0.f, top = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nvec) continue;
        load8(x + t * d + 8 * c, z[i]);
        float wv[8];
        load8(w + 8 * c, wv);
        if (res) {
            float r[8];
            load8_stream(res + t * d + 8 * c, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[i][j] = stored(z[i][j] + r[j], res);
            store8(z_out + t * d + 8 * c, z[i]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            ss = fmaf(z[i][j], z[i][j], ss);
            z[i][j] *= wv[j];
            if (CODES) top = fmaxf(top, fabsf(z[i][j]));
        }
    }
    if (CODES)
        row_reduce(ss, top, red, nwarps);
    else
        ss = row_reduce(ss, red, nwarps);
    const float rstd = 1.0f / sqrtf(ss / (float)d + eps);
    if (rstd_out && threadIdx.x == 0) rstd_out[t] = rstd;
    if (CODES) {
        // rows of values near zero take a power of two out first: 448 / top stays finite
        const float up = top < 1e-30f ? 1.2676506e30f : 1.f;  // 2^100
        const float f = top > 0.f ? __fdiv_rn(448.f, top * up) : 0.f;
        if (threadIdx.x == 0) sy[t] = top > 0.f ? top * rstd / 448.f : 1.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nvec) continue;
            float q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = z[i][j] * up * f;
            *reinterpret_cast<uint2*>(yq + t * d + 8 * c) = codes8_of(q);
        }
    }
    if (!y) return;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nvec) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) z[i][j] *= rstd;
        store8(y + t * d + 8 * c, z[i]);
    }
}

// 16 bytes from global to shared memory, completed by cp_wait of the thread that issued it.
__device__ __forceinline__ void cp16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One row per CTA and step; CTA b takes the rows b, b + gridDim.x, ... Each thread copies its own
// vectors of the next rows to shared memory (STAGES - 1 rows ahead, no barrier: it reads
// only what its own warp copied), so loads stay in flight across the row's reduction. It keeps the
// partial sums of dw for its own columns over all rows, so dw costs no traffic per row: the CTA's
// sums are written once, and norm_dw_kernel adds them in the CTAs' order.
//
// 65,536 x 4096 with norm_dw_kernel: bf16 stream (2.15 GB) 323 us, 0.98 of a copy; fp32 stream with
// the bf16 dx 632 us, 1.00.
template <typename R, int VPT, int STAGES>
__global__ void __launch_bounds__(512) norm_bwd_kernel(
    const __nv_bfloat16* __restrict__ dy, const R* dres, const R* __restrict__ z,
    const float* __restrict__ rstd, const float* __restrict__ w, int64_t T, int d, R* dz,
    __nv_bfloat16* __restrict__ dx, float* __restrict__ part) {
    constexpr int RW = sizeof(R) / 2;  // 16-byte words of a vector of R
    constexpr int SLOTS = VPT * (1 + 2 * RW);
    extern __shared__ __align__(16) uint4 ring[];  // [stage][vector of a thread][dy | z | dres][thread]
    __shared__ float2 red[2][32];
    const int nvec = d / 8, nwarps = blockDim.x / 32, nt = blockDim.x, lane = threadIdx.x % 32;
    auto area = [&](int stage, int i, int which) {  // of dy, z, dres: one, RW and RW words per thread
        return ring + (stage * SLOTS + i * (1 + 2 * RW) + (which == 0 ? 0 : which == 1 ? 1 : 1 + RW)) * nt;
    };
    auto fetch = [&](int64_t t, int stage) {
        if (t < T) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c0 = threadIdx.x - lane + i * nt;  // the warp's first vector
                if (c0 + lane < nvec) cp16(area(stage, i, 0) + threadIdx.x, dy + t * d + 8 * (c0 + lane));
#pragma unroll
                for (int q = 0; q < RW; ++q) {
                    const int word = lane + 32 * q;  // of the warp's vectors: whole lines per copy
                    if (c0 + word / RW >= nvec) continue;
                    const int to = (threadIdx.x - lane) * RW + word;
                    cp16(area(stage, i, 1) + to, reinterpret_cast<const uint4*>(z + t * d + 8 * c0) + word);
                    if (dres)
                        cp16(area(stage, i, 2) + to, reinterpret_cast<const uint4*>(dres + t * d + 8 * c0) + word);
                }
            }
        }
        cp_commit();
    };
    auto value8 = [&](const uint4* a, float (&v)[8]) {  // the thread's vector of R
        if constexpr (RW == 1) {
            load8(reinterpret_cast<const __nv_bfloat16*>(a + threadIdx.x), v);
        } else {
            load8(reinterpret_cast<const float*>(a + 2 * threadIdx.x), v);
        }
    };
    float acc[VPT][8], wv[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * nt;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
        if (c < nvec) load8(w + 8 * c, wv[i]);
    }
#pragma unroll
    for (int q = 0; q < STAGES - 1; ++q) fetch(blockIdx.x + (int64_t)q * gridDim.x, q);
    int side = 0, stage = 0;
    float rs = blockIdx.x < T ? rstd[blockIdx.x] : 0.f;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x, side ^= 1) {
        const int ahead = stage == 0 ? STAGES - 1 : stage - 1;
        __syncwarp();  // the warp is done with that stage's row
        fetch(t + (int64_t)(STAGES - 1) * gridDim.x, ahead);
        cp_wait<STAGES - 1>();
        __syncwarp();  // a thread's vectors of R are copied by its warp
        const float rs_next = t + gridDim.x < T ? rstd[t + gridDim.x] : 0.f;
        float g[VPT][8], h[VPT][8];  // dy w and xhat
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * nt;
            if (c >= nvec) continue;
            load8(reinterpret_cast<const __nv_bfloat16*>(area(stage, i, 0) + threadIdx.x), g[i]);
            value8(area(stage, i, 1), h[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[i][j] *= rs;
                acc[i][j] = fmaf(g[i][j], h[i][j], acc[i][j]);
                g[i][j] *= wv[i][j];
                dot = fmaf(g[i][j], h[i][j], dot);
            }
        }
        dot = row_reduce(dot, red[side], nwarps) / (float)d;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * nt;
            if (c >= nvec) continue;
            float o[8];
            if (dres) {
                value8(area(stage, i, 2), o);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = fmaf(rs, g[i][j] - h[i][j] * dot, o[j]);
            store8(dz + t * d + 8 * c, o);
            if (dx) store8(dx + t * d + 8 * c, o);
        }
        rs = rs_next;
        stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    cp_wait<0>();
    grid_launch_dependents();
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * nt;
        if (c < nvec) put8(part + (int64_t)blockIdx.x * d + 8 * c, acc[i]);
    }
}

// Rows of up to 1024 columns: a warp each, so that a row needs no barrier. The warp copies its own
// next rows ahead and reads a row from shared memory twice, for the dot product and for the
// gradient, instead of holding 64 values a thread across the reduction. The CTA's warps add their
// sums of dw in their order at the end.
//
// 8192 x 1024 bf16 with norm_dw_kernel (67 MB): 15.8 us, 0.63 of a copy (a CTA per row with the ring
// above: 26.5); 16,384 x 1024 fp32 46 us, 0.86; 65,536 x 256 bf16 28 us, 0.71. The launch, the first
// rows' latency and the sums of dw are 4.5 us of each; the rest that short rows lack (3.5 us at 256
// columns) goes by a row's fixed work, with 16 warps per SM to hide it (four CTAs, also where
// registers would let more in).
constexpr int kRowWarps = 4;

template <typename R, int VPT, int STAGES>
__global__ void __launch_bounds__(32 * kRowWarps) norm_bwd_rows_kernel(
    const __nv_bfloat16* __restrict__ dy, const R* dres, const R* __restrict__ z,
    const float* __restrict__ rstd, const float* __restrict__ w, int64_t T, int d, R* dz,
    __nv_bfloat16* __restrict__ dx, float* __restrict__ part) {
    constexpr int RW = sizeof(R) / 2;  // 16-byte words of a vector of R
    constexpr int VW = 1 + 2 * RW;     // of a vector of all three tensors
    extern __shared__ __align__(16) uint4 ring[];  // [warp][stage][vector][dy | z | dres]; then sums of dw
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int nvec = d / 8;
    auto area = [&](int stage, int i, int which) {
        return ring + (((warp * STAGES + stage) * VPT + i) * VW + (which == 0 ? 0 : which == 1 ? 1 : 1 + RW)) * 32;
    };
    auto fetch = [&](int64_t t, int stage) {
        if (t < T) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (lane + 32 * i < nvec) cp16(area(stage, i, 0) + lane, dy + t * d + 8 * (lane + 32 * i));
#pragma unroll
                for (int q = 0; q < RW; ++q) {
                    const int word = lane + 32 * q;  // whole lines per copy
                    if (32 * i + word / RW >= nvec) continue;
                    const int64_t at = t * d + 256 * i;
                    cp16(area(stage, i, 1) + word, reinterpret_cast<const uint4*>(z + at) + word);
                    if (dres) cp16(area(stage, i, 2) + word, reinterpret_cast<const uint4*>(dres + at) + word);
                }
            }
        }
        cp_commit();
    };
    auto value8 = [&](const uint4* a, float (&v)[8]) {  // the lane's vector of R
        if constexpr (RW == 1) {
            load8(reinterpret_cast<const __nv_bfloat16*>(a + lane), v);
        } else {
            load8(reinterpret_cast<const float*>(a + 2 * lane), v);
        }
    };
    const int64_t first = (int64_t)blockIdx.x * kRowWarps + warp, stride = (int64_t)gridDim.x * kRowWarps;
#pragma unroll
    for (int q = 0; q < STAGES - 1; ++q) fetch(first + q * stride, q);
    float acc[VPT][8], wv[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = lane + 32 * i;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = wv[i][j] = 0.f;
        if (c < nvec) load8(w + 8 * c, wv[i]);
    }
    const float inv_d = 1.0f / (float)d;
    int stage = 0;
    float rs = first < T ? rstd[first] : 0.f;
    for (int64_t t = first; t < T; t += stride) {
        const int ahead = stage == 0 ? STAGES - 1 : stage - 1;
        __syncwarp();  // every lane is done with that stage's row
        fetch(t + (STAGES - 1) * stride, ahead);
        cp_wait<STAGES - 1>();
        __syncwarp();
        const float rs_next = t + stride < T ? rstd[t + stride] : 0.f;
        float dot = 0.f;  // of dy w and z: rstd comes after the sum
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (lane + 32 * i >= nvec) continue;
            float g[8], h[8];
            load8(reinterpret_cast<const __nv_bfloat16*>(area(stage, i, 0) + lane), g);
            value8(area(stage, i, 1), h);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float p = g[j] * h[j];
                acc[i][j] = fmaf(p, rs, acc[i][j]);
                dot = fmaf(p, wv[i][j], dot);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        const float c1 = -(dot * rs) * inv_d * rs;  // dz = rs (dy w + c1 z) + dres
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + 32 * i;
            if (c >= nvec) continue;
            float g[8], h[8], o[8];
            load8(reinterpret_cast<const __nv_bfloat16*>(area(stage, i, 0) + lane), g);
            value8(area(stage, i, 1), h);
            if (dres) {
                value8(area(stage, i, 2), o);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = fmaf(fmaf(c1, h[j], g[j] * wv[i][j]), rs, o[j]);
            store8(dz + t * d + 8 * c, o);
            if (dx) store8(dx + t * d + 8 * c, o);
        }
        rs = rs_next;
        stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    cp_wait<0>();
    grid_launch_dependents();
    __syncthreads();  // the rings are done with
    float* const sums = reinterpret_cast<float*>(ring);  // [warp][d]
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (lane + 32 * i < nvec) put8(sums + warp * d + 8 * (lane + 32 * i), acc[i]);
    __syncthreads();
    for (int j = threadIdx.x; j < d; j += 32 * kRowWarps) {
        float a = sums[j];
#pragma unroll
        for (int q = 1; q < kRowWarps; ++q) a += sums[q * d + j];
        part[(int64_t)blockIdx.x * d + j] = a;
    }
}

// Rows of more than 8192 columns, which no layer here has: the same sums, with plain loads and up to
// 1024 threads. A row's second reading comes from L2, and its dw sums are read and written there
// too, 8 bytes an element for every row: 8192 x 16,384 bf16 takes 265 us, 0.60 of a copy. (A ring of two
// bf16 rows would fit up to 16,384 columns, with the sums in registers; it is not built.)
template <typename R, int VPT>
__global__ void __launch_bounds__(1024) norm_bwd_wide_kernel(
    const __nv_bfloat16* __restrict__ dy, const R* dres, const R* __restrict__ z,
    const float* __restrict__ rstd, const float* __restrict__ w, int64_t T, int d, R* dz,
    __nv_bfloat16* __restrict__ dx, float* __restrict__ part) {
    __shared__ float2 red[2][32];
    const int nvec = d / 8, nwarps = blockDim.x / 32;
    float* sums = part + (int64_t)blockIdx.x * d;  // the CTA's own row, in global memory
    int side = 0;
    bool begun = false;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x, side ^= 1, begun = true) {
        const float rs = rstd[t];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nvec) continue;
            float g[8], h[8], wv[8], a[8];
            load8(dy + t * d + 8 * c, g);
            load8_stream(z + t * d + 8 * c, h);
            load8(w + 8 * c, wv);
            if (begun) load8(sums + 8 * c, a);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[j] *= rs;
                a[j] = fmaf(g[j], h[j], begun ? a[j] : 0.f);
                dot = fmaf(g[j] * wv[j], h[j], dot);
            }
            put8(sums + 8 * c, a);
        }
        dot = row_reduce(dot, red[side], nwarps) / (float)d;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nvec) continue;
            float g[8], h[8], wv[8], o[8];
            load8(dy + t * d + 8 * c, g);
            load8_stream(z + t * d + 8 * c, h);
            load8(w + 8 * c, wv);
            if (dres) {
                load8_stream(dres + t * d + 8 * c, o);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = fmaf(rs, g[j] * wv[j] - h[j] * rs * dot, o[j]);
            store8(dz + t * d + 8 * c, o);
            if (dx) store8(dx + t * d + 8 * c, o);
        }
    }
}

// dw[j] = sum of part[r][j] over r < rows: blocks of 32 columns (eight 16-byte vectors) x 128 row
// strands, each strand summed in order, then the strands by a tree. The few rows of a strand
// are loaded together: the launch is all latency (4.5 us alone, about half of it behind the kernel
// before, whose last CTAs it waits for).
constexpr int kDwStrands = 128;

__global__ void __launch_bounds__(8 * kDwStrands) norm_dw_kernel(const float* __restrict__ part, int rows,
                                                                 int d, float* __restrict__ dw) {
    constexpr int N = (kNormBwdParts + kDwStrands - 1) / kDwStrands;
    __shared__ float s[kDwStrands][33];
    const int tx = threadIdx.x % 8, ty = threadIdx.x / 8;
    const int j = blockIdx.x * 32 + 4 * tx;
    float4 v[N];
    grid_dependency_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = ty + i * kDwStrands;
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows && j < d)  // d is a multiple of 8
            v[i] = *reinterpret_cast<const float4*>(part + (int64_t)r * d + j);
    }
    float4 a = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) a.x += v[i].x, a.y += v[i].y, a.z += v[i].z, a.w += v[i].w;
    s[ty][4 * tx] = a.x, s[ty][4 * tx + 1] = a.y, s[ty][4 * tx + 2] = a.z, s[ty][4 * tx + 3] = a.w;
    __syncthreads();
    // a warp per column: four strands a lane, then the lanes by a butterfly
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < kDwStrands / 32; ++q) t += s[lane + 32 * q][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0 && blockIdx.x * 32 + warp < d) dw[blockIdx.x * 32 + warp] = t;
}
static_assert(8 * kDwStrands == 32 * 32, "a warp per column");

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

struct NormShape {
    int threads, vpt;
};

// Threads of one row and vectors of eight values per thread (1, 2 or 4). Many rows: four vectors
// each, so that few threads share the reduction's and the row's fixed work (8191 x 1024: 13.6 us
// at a warp a row, 14.1 at 128 threads). Few rows, where a row's latency counts: as many threads
// as there are vectors (one row of 4096 with codes: 2.4 us, 2.6 at two vectors each).
NormShape norm_shape(int64_t T, int d) {
    const int nvec = d / 8;
    int vpt = 1;
    if (T >= 2 * (int64_t)sm_count())
        while (vpt < 4 && 32 * vpt < nvec) vpt *= 2;
    else
        while (vpt < 4 && 1024 * vpt < nvec) vpt *= 2;
    return {(int)cdiv(cdiv(nvec, vpt), 32) * 32, vpt};
}

template <typename R>
int launch_norm_fwd(const moe_bf16* x, const void* res, const float* w, float eps, int64_t T, int d,
                    void* z_out, moe_bf16* y, uint8_t* yq, float* sy, float* rstd,
                    cudaStream_t st) {
    const NormShape s = norm_shape(T, d);
    const int rows = s.threads == 32 ? 4 : 1;
    const dim3 block(s.threads, rows);
    const unsigned grid = (unsigned)cdiv(T, rows);
    auto go = [&](auto kern) {
        kern<<<grid, block, 0, st>>>(reinterpret_cast<const __nv_bfloat16*>(x),
                                     static_cast<const R*>(res), w, eps, T, d,
                                     static_cast<R*>(z_out), reinterpret_cast<__nv_bfloat16*>(y),
                                     yq, sy, rstd);
    };
    if (s.vpt == 1) yq ? go(norm_fwd_kernel<R, 1, true>) : go(norm_fwd_kernel<R, 1, false>);
    else if (s.vpt == 2) yq ? go(norm_fwd_kernel<R, 2, true>) : go(norm_fwd_kernel<R, 2, false>);
    else yq ? go(norm_fwd_kernel<R, 4, true>) : go(norm_fwd_kernel<R, 4, false>);
    return launch_status();
}

constexpr size_t kRingBytes = 104 * 1024;  // the deepest ring that leaves room for two CTAs per SM

template <typename R, int VPT>
int launch_bwd_rows(const __nv_bfloat16* dy, const R* dres, const R* z, const float* rstd, const float* w,
                    int64_t T, int d, R* dz, __nv_bfloat16* dx, float* part, int* rows, cudaStream_t st) {
    constexpr int STAGES = 3;
    size_t smem = (size_t)kRowWarps * STAGES * VPT * (1 + sizeof(R)) * 32 * 16;
    const size_t sums = (size_t)kRowWarps * d * sizeof(float);
    if (sums > smem) smem = sums;
    auto kern = norm_bwd_rows_kernel<R, VPT, STAGES>;
    if (smem > 40 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return MOE_ERR_LAUNCH;
    int64_t ctas = (size_t)(224 * 1024) / (smem + 1024);  // per SM
    if (ctas > 4) ctas = 4;
    *rows = (int)norm_bwd_parts(cdiv(T, kRowWarps));
    if (*rows > ctas * sm_count()) *rows = (int)(ctas * sm_count());
    kern<<<*rows, 32 * kRowWarps, smem, st>>>(dy, dres, z, rstd, w, T, d, dz, dx, part);
    return launch_status();
}

template <typename R, int VPT, int STAGES>
int launch_bwd(const __nv_bfloat16* dy, const R* dres, const R* z, const float* rstd, const float* w,
               int64_t T, int d, int threads, R* dz, __nv_bfloat16* dx, float* part, int* rows,
               cudaStream_t st) {
    const size_t smem = (size_t)STAGES * VPT * (1 + sizeof(R)) * 16 * threads;
    auto kern = norm_bwd_kernel<R, VPT, STAGES>;
    if (smem > 40 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return MOE_ERR_LAUNCH;
    int64_t ctas = (size_t)(224 * 1024) / (smem + 1280);  // per SM
    if (ctas < 1) ctas = 1;
    if (ctas > 4) ctas = 4;
    *rows = (int)norm_bwd_parts(T);
    if (*rows > ctas * sm_count()) *rows = (int)(ctas * sm_count());
    kern<<<*rows, threads, smem, st>>>(dy, dres, z, rstd, w, T, d, dz, dx, part);
    return launch_status();
}

template <typename R>
int launch_norm_bwd(const moe_bf16* dy_, const void* dres_, const void* z_, const float* rstd,
                    const float* w, int64_t T, int d, void* dz_, moe_bf16* dx_, float* part,
                    float* dw, cudaStream_t st) {
    auto* dy = reinterpret_cast<const __nv_bfloat16*>(dy_);
    auto* dx = reinterpret_cast<__nv_bfloat16*>(dx_);
    auto *dres = static_cast<const R*>(dres_), *z = static_cast<const R*>(z_);
    auto* dz = static_cast<R*>(dz_);
    const int nvec = d / 8;
    int rc, rows = 0;
    using std::integral_constant;
    if (nvec <= 128) {
        rc = nvec <= 32   ? launch_bwd_rows<R, 1>(dy, dres, z, rstd, w, T, d, dz, dx, part, &rows, st)
             : nvec <= 64 ? launch_bwd_rows<R, 2>(dy, dres, z, rstd, w, T, d, dz, dx, part, &rows, st)
                          : launch_bwd_rows<R, 4>(dy, dres, z, rstd, w, T, d, dz, dx, part, &rows, st);
    } else if (nvec <= 1024) {
        const int threads = (int)cdiv(cdiv(nvec, 2), 32) * 32;
        const bool deep = 4 * 2 * (1 + sizeof(R)) * 16 * threads <= kRingBytes;
        auto go = [&](auto stages) {
            return launch_bwd<R, 2, decltype(stages)::value>(dy, dres, z, rstd, w, T, d, threads, dz, dx,
                                                             part, &rows, st);
        };
        rc = deep ? go(integral_constant<int, 4>()) : go(integral_constant<int, 2>());
    } else {
        rows = (int)norm_bwd_parts(T);
        norm_bwd_wide_kernel<R, 4><<<rows, (unsigned)cdiv(cdiv(nvec, 4), 32) * 32, 0, st>>>(
            dy, dres, z, rstd, w, T, d, dz, dx, part);
        rc = launch_status();
    }
    if (rc != MOE_OK) return rc;
    return launch_dependent(norm_dw_kernel, dim3((unsigned)cdiv(d, 32)), dim3(8 * kDwStrands), 0, st,
                            (const float*)part, rows, d, dw);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_rms_norm(const moe_bf16* x, const void* residual, int res_type, const float* w,
                            float eps, int64_t T, int d, void* z, moe_bf16* y, uint8_t* yq,
                            float* sy, float* rstd, moe_stream_t stream) {
    if (!x || !w || (!y && !yq)) return MOE_ERR_INVALID_ARG;
    if ((residual == nullptr) != (z == nullptr)) return MOE_ERR_INVALID_ARG;
    if ((yq == nullptr) != (sy == nullptr)) return MOE_ERR_INVALID_ARG;
    if (T <= 0 || d <= 0 || !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
    if (res_type != MOE_TYPE_BF16 && res_type != MOE_TYPE_F32) return MOE_ERR_INVALID_ARG;
    if (d % 8 != 0 || d > kNormMaxD || T > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    for (const void* p : {(const void*)x, residual, (const void*)w, (const void*)z, (const void*)y})
        if (p && !aligned16(p)) return MOE_ERR_INVALID_ARG;
    if (yq && (reinterpret_cast<uintptr_t>(yq) & 7u)) return MOE_ERR_INVALID_ARG;
    if (res_type == MOE_TYPE_F32 && (!aligned32(residual) || !aligned32(z))) return MOE_ERR_INVALID_ARG;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    cudaStream_t st = (cudaStream_t)stream;
    return res_type == MOE_TYPE_F32
               ? launch_norm_fwd<float>(x, residual, w, eps, T, d, z, y, yq, sy, rstd, st)
               : launch_norm_fwd<__nv_bfloat16>(x, residual, w, eps, T, d, z, y, yq, sy, rstd, st);
}

extern "C" int moe_rms_norm_bwd(const moe_bf16* dy, const void* dres, const void* z, int res_type,
                                const float* rstd, const float* w, int64_t T, int d, void* dz,
                                moe_bf16* dx, float* dw, void* ws, size_t ws_bytes,
                                moe_stream_t stream) {
    if (!dy || !z || !rstd || !w || !dz || !dw) return MOE_ERR_INVALID_ARG;
    if (T <= 0 || d <= 0) return MOE_ERR_INVALID_ARG;
    if (res_type != MOE_TYPE_BF16 && res_type != MOE_TYPE_F32) return MOE_ERR_INVALID_ARG;
    if (d % 8 != 0 || d > kNormMaxD || T > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    for (const void* p : {(const void*)dy, dres, z, (const void*)w, (const void*)dz, (const void*)dx})
        if (p && !aligned16(p)) return MOE_ERR_INVALID_ARG;
    if (res_type == MOE_TYPE_F32 && (!aligned32(dres) || !aligned32(z) || !aligned32(dz))) return MOE_ERR_INVALID_ARG;
    if (!ws || !aligned16(ws)) return MOE_ERR_WORKSPACE;
    WsCarver wc(ws, ws_bytes);
    float* part = wc.take<float>((size_t)norm_bwd_parts(T) * d);
    if (!wc.ok()) return MOE_ERR_WORKSPACE;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    cudaStream_t st = (cudaStream_t)stream;
    return res_type == MOE_TYPE_F32
               ? launch_norm_bwd<float>(dy, dres, z, rstd, w, T, d, dz, dx, part, dw, st)
               : launch_norm_bwd<__nv_bfloat16>(dy, dres, z, rstd, w, T, d, dz, dx, part, dw, st);
}
