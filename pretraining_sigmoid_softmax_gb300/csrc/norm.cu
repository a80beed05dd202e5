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
#include <cuda_runtime.h>

#include "common.cuh"
#include "fp8.cuh"
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

// Codes of eight values under the row's scale. The division-free quotient holds while neither
// the scale nor its reciprocal leaves the normal range; rows of values near the type's ends
// (|y| below about 1e-27, or infinite) divide.
__device__ __forceinline__ uint2 row_codes(const float (&v)[8], const Fp8Scale& sc) {
    if (sc.s > 1e-30f && sc.s < 1e30f) return codes8f(v, sc);
    uint32_t packed[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const __nv_fp8_storage_t q =
            __nv_cvt_float_to_fp8(__fdiv_rn(v[j], sc.s), __NV_SATFINITE, __NV_E4M3);
        packed[j / 4] |= (uint32_t)q << (8 * (j % 4));
    }
    return make_uint2(packed[0], packed[1]);
}

struct SumOp {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct MaxOp {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// The value over all threads of a row, in a fixed order: a butterfly within each warp, then
// (rows of several warps) the warps' values from shared memory in their order. `red` is one
// slot per warp, written by no later reduction before a barrier has passed.
template <typename Op>
__device__ __forceinline__ float row_reduce(float v, float* red, int nwarps, Op op) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (nwarps == 1) return v;  // rows of one warp: no barrier
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    float r = red[0];
    for (int i = 1; i < nwarps; ++i) r = op(r, red[i]);
    return r;
}

// blockDim = (threads per row, rows per CTA); rows of one warp may share a CTA. Thread i of a
// row owns its vectors i, i + blockDim.x, ... (eight values each), VPT of them at most.
template <typename R, int VPT>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(
    const __nv_bfloat16* x, const R* res, const float* __restrict__ w, float eps, int64_t T, int d,
    R* z_out, __nv_bfloat16* y, uint8_t* __restrict__ yq, float* __restrict__ sy,
    float* __restrict__ rstd_out) {
    __shared__ float red[2][32];
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= T) return;  // a whole row (a warp of its own where rows share a CTA)
    const int nvec = d / 8, nwarps = blockDim.x / 32;
    float z[VPT][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nvec) {
#pragma unroll
            for (int j = 0; j < 8; ++j) z[i][j] = 0.f;
            continue;
        }
        load8(x + t * d + 8 * c, z[i]);
        if (res) {
            float r[8];
            load8(res + t * d + 8 * c, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[i][j] = stored(z[i][j] + r[j], res);
            store8(z_out + t * d + 8 * c, z[i]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(z[i][j], z[i][j], ss);
    }
    ss = row_reduce(ss, red[0], nwarps, SumOp());
    const float rstd = 1.0f / sqrtf(ss / (float)d + eps);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nvec) continue;
        float wv[8];
        load8(w + 8 * c, wv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            z[i][j] = z[i][j] * rstd * wv[j];
            amax = fmaxf(amax, fabsf(z[i][j]));
        }
        if (y) store8(y + t * d + 8 * c, z[i]);
    }
    if (rstd_out && threadIdx.x == 0) rstd_out[t] = rstd;
    if (!yq) return;
    amax = row_reduce(amax, red[1], nwarps, MaxOp());
    const Fp8Scale sc(amax);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < nvec) *reinterpret_cast<uint2*>(yq + t * d + 8 * c) = row_codes(z[i], sc);
    }
    if (threadIdx.x == 0) sy[t] = sc.s;
}

// One row per CTA and step; CTA b takes the rows b, b + gridDim.x, ... Each thread keeps the
// partial sums of dw for its own columns over all of them, so dw costs no traffic per row: the
// CTA's sums are written once, and norm_dw_kernel adds them in the CTAs' order.
template <typename R, int VPT>
__global__ void __launch_bounds__(1024) norm_bwd_kernel(
    const __nv_bfloat16* __restrict__ dy, const R* dres, const R* __restrict__ z,
    const float* __restrict__ rstd, const float* __restrict__ w, int64_t T, int d, R* dz,
    __nv_bfloat16* __restrict__ dx, float* __restrict__ part) {
    __shared__ float red[2][32];
    const int nvec = d / 8, nwarps = blockDim.x / 32;
    float acc[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    int side = 0;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x, side ^= 1) {
        const float rs = rstd[t];
        float g[VPT][8], h[VPT][8];  // dy w and xhat
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nvec) continue;
            float wv[8];
            load8(dy + t * d + 8 * c, g[i]);
            load8(z + t * d + 8 * c, h[i]);
            load8(w + 8 * c, wv);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[i][j] *= rs;
                acc[i][j] = fmaf(g[i][j], h[i][j], acc[i][j]);
                g[i][j] *= wv[j];
                dot = fmaf(g[i][j], h[i][j], dot);
            }
        }
        dot = row_reduce(dot, red[side], nwarps, SumOp()) / (float)d;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nvec) continue;
            float o[8];
            if (dres)
                load8(dres + t * d + 8 * c, o);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = fmaf(rs, g[i][j] - h[i][j] * dot, o[j]);
            store8(dz + t * d + 8 * c, o);
            if (dx) store8(dx + t * d + 8 * c, o);
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < nvec) store8(part + (int64_t)blockIdx.x * d + 8 * c, acc[i]);
    }
}

// dw[j] = sum of part[r][j] over r < rows: blocks of 32 columns x 8 row strands, each strand
// summed in order, then the strands in order.
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* __restrict__ part, int rows,
                                                      int d, float* __restrict__ dw) {
    __shared__ float s[8][33];
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    const int j = blockIdx.x * 32 + tx;
    float a = 0.f;
    if (j < d)
        for (int r = ty; r < rows; r += 8) a += part[(int64_t)r * d + j];
    s[ty][tx] = a;
    __syncthreads();
    if (ty == 0 && j < d) {
#pragma unroll
        for (int q = 1; q < 8; ++q) a += s[q][tx];
        dw[j] = a;
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

template <typename R>
int launch_norm_bwd(const moe_bf16* dy, const void* dres, const void* z, const float* rstd,
                    const float* w, int64_t T, int d, void* dz, moe_bf16* dx, float* part,
                    float* dw, cudaStream_t st) {
    const NormShape s = norm_shape(d);
    const int64_t rows = norm_bwd_parts(T);
    auto go = [&](auto kern) {
        kern<<<(unsigned)rows, s.threads, 0, st>>>(
            reinterpret_cast<const __nv_bfloat16*>(dy), static_cast<const R*>(dres),
            static_cast<const R*>(z), rstd, w, T, d, static_cast<R*>(dz),
            reinterpret_cast<__nv_bfloat16*>(dx), part);
    };
    if (s.vpt == 1) go(norm_bwd_kernel<R, 1>);
    else if (s.vpt == 2) go(norm_bwd_kernel<R, 2>);
    else go(norm_bwd_kernel<R, 4>);
    if (launch_status() != MOE_OK) return MOE_ERR_LAUNCH;
    norm_dw_kernel<<<(unsigned)cdiv(d, 32), 256, 0, st>>>(part, (int)rows, d, dw);
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
