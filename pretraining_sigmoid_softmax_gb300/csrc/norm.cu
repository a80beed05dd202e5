// Residual addition and root-mean-square norm in front of the MoE layer, and its backward.
//
// Forward, per token: z = residual + x (rounded to the residual stream's type), rstd =
// 1 / sqrt(mean(z^2) + eps), y = z rstd w; y leaves as bf16 and, for the FP8 experts, as E4M3
// codes under one scale per row (amax / 448 of the unrounded y, 1 for a zero row).
// Backward, with xhat = z rstd and g = dy w: dz = rstd (g - xhat mean(g xhat)) + dres,
// dw = sum over tokens of dy xhat.
//
// Both are bound by HBM: every tensor is read or written once. A row stays in registers
// between its loads and its stores.
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

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
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

__device__ __forceinline__ float row_reduce(float s, float* red, int nwarps) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (nwarps == 1) return s;
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = s;
    __syncthreads();
    s = red[0];
    for (int i = 1; i < nwarps; ++i) s += red[i];
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
template <typename R, int VPT>
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
            load8(res + t * d + 8 * c, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[i][j] = stored(z[i][j] + r[j], res);
            store8(z_out + t * d + 8 * c, z[i]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            ss = fmaf(z[i][j], z[i][j], ss);
            z[i][j] *= wv[j];
            top = fmaxf(top, fabsf(z[i][j]));
        }
    }
    row_reduce(ss, top, red, nwarps);
    const float rstd = 1.0f / sqrtf(ss / (float)d + eps);
    if (rstd_out && threadIdx.x == 0) rstd_out[t] = rstd;
    if (yq) {
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
// only what it copied itself), so loads stay in flight across the row's reduction. It keeps the
// partial sums of dw for its own columns over all rows, so dw costs no traffic per row: the CTA's
// sums are written once, and norm_dw_kernel adds them in the CTAs' order.
template <typename R, int VPT, int STAGES>
__global__ void __launch_bounds__(VPT == 1 ? 256 : 512) norm_bwd_kernel(
    const __nv_bfloat16* __restrict__ dy, const R* dres, const R* __restrict__ z,
    const float* __restrict__ rstd, const float* __restrict__ w, int64_t T, int d, R* dz,
    __nv_bfloat16* __restrict__ dx, float* __restrict__ part) {
    constexpr int RW = sizeof(R) / 2;  // 16-byte words of a vector of R
    constexpr int SLOTS = VPT * (1 + 2 * RW);
    extern __shared__ __align__(16) uint4 ring[];  // [stage][slot][thread]
    __shared__ float red[2][32];
    const int nvec = d / 8, nwarps = blockDim.x / 32, nt = blockDim.x;
    auto slot = [&](int stage, int k) { return ring + ((stage * SLOTS + k) * nt + threadIdx.x); };
    auto fetch = [&](int64_t t, int stage) {
        if (t < T) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = threadIdx.x + i * nt;
                if (c >= nvec) continue;
                const int64_t at = t * d + 8 * c;
                const int k = i * (1 + 2 * RW);
                cp16(slot(stage, k), dy + at);
#pragma unroll
                for (int q = 0; q < RW; ++q) {
                    cp16(slot(stage, k + 1 + q), reinterpret_cast<const uint4*>(z + at) + q);
                    if (dres) cp16(slot(stage, k + 1 + RW + q), reinterpret_cast<const uint4*>(dres + at) + q);
                }
            }
        }
        cp_commit();
    };
    auto value8 = [&](int stage, int k, auto* type, float (&v)[8]) {
        using S = std::remove_pointer_t<decltype(type)>;
        if constexpr (sizeof(S) == 2) {
            load8(reinterpret_cast<const S*>(slot(stage, k)), v);
        } else {
            const float4 a = *reinterpret_cast<const float4*>(slot(stage, k));
            const float4 b = *reinterpret_cast<const float4*>(slot(stage, k + 1));
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
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
        fetch(t + (int64_t)(STAGES - 1) * gridDim.x, ahead);
        cp_wait<STAGES - 1>();
        const float rs_next = t + gridDim.x < T ? rstd[t + gridDim.x] : 0.f;
        float g[VPT][8], h[VPT][8];  // dy w and xhat
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * nt;
            if (c >= nvec) continue;
            value8(stage, i * (1 + 2 * RW), (__nv_bfloat16*)nullptr, g[i]);
            value8(stage, i * (1 + 2 * RW) + 1, (R*)nullptr, h[i]);
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
                value8(stage, i * (1 + 2 * RW) + 1 + RW, (R*)nullptr, o);
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
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * nt;
        if (c < nvec) store8(part + (int64_t)blockIdx.x * d + 8 * c, acc[i]);
    }
}

// Rows too wide for the ring: the same sums, with plain loads and up to 1024 threads.
template <typename R, int VPT>
__global__ void __launch_bounds__(1024) norm_bwd_wide_kernel(
    const __nv_bfloat16* __restrict__ dy, const R* dres, const R* __restrict__ z,
    const float* __restrict__ rstd, const float* __restrict__ w, int64_t T, int d, R* dz,
    __nv_bfloat16* __restrict__ dx, float* __restrict__ part) {
    __shared__ float red[2][32];
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
            load8(z + t * d + 8 * c, h);
            load8(w + 8 * c, wv);
            if (begun) load8(sums + 8 * c, a);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[j] *= rs;
                a[j] = fmaf(g[j], h[j], begun ? a[j] : 0.f);
                dot = fmaf(g[j] * wv[j], h[j], dot);
            }
            store8(sums + 8 * c, a);
        }
        dot = row_reduce(dot, red[side], nwarps) / (float)d;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nvec) continue;
            float g[8], h[8], wv[8], o[8];
            load8(dy + t * d + 8 * c, g);
            load8(z + t * d + 8 * c, h);
            load8(w + 8 * c, wv);
            if (dres) {
                load8(dres + t * d + 8 * c, o);
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

// dw[j] = sum of part[r][j] over r < rows: blocks of 32 columns (eight 16-byte vectors) x 32 row
// strands, each strand summed in order, then the strands in order.
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* __restrict__ part, int rows,
                                                      int d, float* __restrict__ dw) {
    __shared__ float s[32][33];
    const int tx = threadIdx.x % 8, ty = threadIdx.x / 8;
    const int j = blockIdx.x * 32 + 4 * tx;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (j < d) {  // d is a multiple of 8
#pragma unroll 4
        for (int r = ty; r < rows; r += 32) {
            const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)r * d + j);
            a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
        }
    }
    s[ty][4 * tx] = a.x, s[ty][4 * tx + 1] = a.y, s[ty][4 * tx + 2] = a.z, s[ty][4 * tx + 3] = a.w;
    __syncthreads();
    if (threadIdx.x < 32 && blockIdx.x * 32 + threadIdx.x < d) {
        float t = 0.f;
#pragma unroll
        for (int q = 0; q < 32; ++q) t += s[q][threadIdx.x];
        dw[blockIdx.x * 32 + threadIdx.x] = t;
    }
}

struct NormShape {
    int threads, vpt;
};

// Threads of one row, and vectors of eight values per thread.
NormShape norm_shape(int d) {
    const int nvec = d / 8;
    const int vpt = nvec <= 256 ? 1 : nvec <= 1024 ? 2 : 4;
    return {(int)cdiv(cdiv(nvec, vpt), 32) * 32, vpt};
}

template <typename R>
int launch_norm_fwd(const moe_bf16* x, const void* res, const float* w, float eps, int64_t T, int d,
                    void* z_out, moe_bf16* y, uint8_t* yq, float* sy, float* rstd,
                    cudaStream_t st) {
    const NormShape s = norm_shape(d);
    const int rows = s.threads == 32 ? 8 : 1;
    const dim3 block(s.threads, rows);
    const unsigned grid = (unsigned)cdiv(T, rows);
    auto go = [&](auto kern) {
        kern<<<grid, block, 0, st>>>(reinterpret_cast<const __nv_bfloat16*>(x),
                                     static_cast<const R*>(res), w, eps, T, d,
                                     static_cast<R*>(z_out), reinterpret_cast<__nv_bfloat16*>(y),
                                     yq, sy, rstd);
    };
    if (s.vpt == 1) go(norm_fwd_kernel<R, 1>);
    else if (s.vpt == 2) go(norm_fwd_kernel<R, 2>);
    else go(norm_fwd_kernel<R, 4>);
    return launch_status();
}

constexpr size_t kRingBytes = 104 * 1024;  // the deepest ring that leaves room for two CTAs per SM

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
    const NormShape s = norm_shape(d);
    const size_t row = (size_t)s.vpt * (1 + sizeof(R)) * 16 * s.threads;  // ring bytes of one row
    int rc, rows = 0;
    if (s.vpt == 4) {
        rows = (int)norm_bwd_parts(T);
        norm_bwd_wide_kernel<R, 4><<<rows, s.threads, 0, st>>>(dy, dres, z, rstd, w, T, d, dz, dx, part);
        rc = launch_status();
    } else {
        auto go = [&](auto vpt, auto stages) {
            return launch_bwd<R, decltype(vpt)::value, decltype(stages)::value>(
                dy, dres, z, rstd, w, T, d, s.threads, dz, dx, part, &rows, st);
        };
        const bool deep = 4 * row <= kRingBytes;
        using std::integral_constant;
        if (s.vpt == 1)
            rc = deep ? go(integral_constant<int, 1>(), integral_constant<int, 4>())
                      : go(integral_constant<int, 1>(), integral_constant<int, 2>());
        else
            rc = deep ? go(integral_constant<int, 2>(), integral_constant<int, 4>())
                      : go(integral_constant<int, 2>(), integral_constant<int, 2>());
    }
    if (rc != MOE_OK) return rc;
    norm_dw_kernel<<<(unsigned)cdiv(d, 32), 256, 0, st>>>(part, rows, d, dw);
    return launch_status();
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
