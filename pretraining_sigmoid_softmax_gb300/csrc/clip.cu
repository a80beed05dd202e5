// Global norm over a step's gradients, and their clipping.
//
// norm = sqrt(sum over all tensors of the sum of squares); coef = max_norm / norm where the
// norm is finite and above max_norm, else 1; out = coef * gradient. The tensors are described
// to the kernels by a table in the launch's parameters (no device copy of it, so a captured
// launch keeps its own), cut into chunks that the CTAs share.
//
// Bound by HBM: every gradient is read once for the norm and once more for the scaled copy, since
// the factor is known only after the last element. 2.4 GB of gradients (an expert layer's of 64
// x 1536 x 4096): 1.10 to 1.13 ms, 0.95 to 0.97 of a copy's rate for the three passes (7.25 GB). A
// short list is all latency: six tensors of 0.8 M elements, 7.3 us in two launches.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <new>
#include <type_traits>
#include <vector>

#include "common.cuh"
#include "sizes.h"

namespace moe {
namespace {

constexpr int kClipThreads = 512;
constexpr int kChunk = 16384;  // elements: 32 per thread (8 are slower even for 0.8 M: 9.2 us, not 7.2)

struct ClipEntry {
    const void* g;
    void* out;
    int64_t n;
    int32_t first;  // chunk number of the tensor's first chunk
    int32_t type;
};

// A launch's tensors. The small table keeps a short list's launch short; kernel parameters
// hold 32,764 bytes at most.
template <int N>
struct ClipTable {
    ClipEntry t[N];
    int32_t count;
    int32_t chunks;
};
constexpr int kSmallTable = 32;
constexpr int kLargeTable = 960;
static_assert(sizeof(ClipTable<kLargeTable>) <= 32000, "kernel parameters");

// Elements before the first 16-byte boundary.
template <typename S>
__device__ __forceinline__ int64_t head_of(const void* p, int64_t n) {
    const int64_t h = (int64_t)((16u - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / (int64_t)sizeof(S);
    return h < n ? h : n;
}

__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16* p) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f(float v, float* p) { *p = v; }

template <typename S> struct Vec;
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static __forceinline__ void get(uint4 u, float (&v)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[2 * q] = bf16_lo(w[q]);
            v[2 * q + 1] = bf16_hi(w[q]);
        }
    }
    __device__ static __forceinline__ uint4 put(const float (&v)[8]) {
        return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                          pack_bf16x2(v[6], v[7]));
    }
    static constexpr uint32_t kMagnitude = 0x7fff7fffu;
};
template <> struct Vec<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ void get(uint4 u, float (&v)[4]) {
        v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y);
        v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
    }
    __device__ static __forceinline__ uint4 put(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                          __float_as_uint(v[3]));
    }
    static constexpr uint32_t kMagnitude = 0x7fffffffu;
};

// Squares of up to four vectors. They are summed in fp32 where that holds them: a sum within
// [2^-100, FLT_MAX] lost less than 2^-44 of itself to squares below the subnormal range and
// nothing to overflow. Any other sum that is not of zeros alone is formed again in 64 bits.
template <typename S>
__device__ __forceinline__ double squares(const uint4 (&u)[4]) {
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float v[Vec<S>::N];
        Vec<S>::get(u[q], v);
#pragma unroll
        for (int j = 0; j < Vec<S>::N; ++j) s = fmaf(v[j], v[j], s);
    }
    if (s >= 7.8886e-31f && s <= 3.4028234e38f) return (double)s;
    uint32_t any = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) any |= (u[q].x | u[q].y | u[q].z | u[q].w) & Vec<S>::kMagnitude;
    if (any == 0) return 0.0;
    double d = 0.0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float v[Vec<S>::N];
        Vec<S>::get(u[q], v);
#pragma unroll
        for (int j = 0; j < Vec<S>::N; ++j) d = fma((double)v[j], (double)v[j], d);
    }
    return d;
}

// Walks the elements [lo, hi) of a tensor whose first 16-byte boundary is at element `head`:
// f4(first element, vectors) for groups of four vectors per thread, f1(element) for the rest.
template <typename S, typename F1, typename F4>
__device__ __forceinline__ void walk(const S* g, int64_t n, int64_t c, F1&& f1, F4&& f4) {
    constexpr int N = Vec<S>::N;
    const int64_t head = head_of<S>(g, n);
    const int64_t lo = c * kChunk, hi = min(n - head, lo + kChunk);  // past the head
    if (c == 0 && threadIdx.x < head) f1((int64_t)threadIdx.x);
    const int64_t full = lo + (hi - lo) / N * N;
    const int64_t stride = (int64_t)kClipThreads * N;
    for (int64_t i0 = lo + (int64_t)threadIdx.x * N; i0 < full; i0 += 4 * stride) {
        uint4 u[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            u[q] = make_uint4(0, 0, 0, 0);
            if (i0 + q * stride < full)
                u[q] = *reinterpret_cast<const uint4*>(g + head + i0 + q * stride);
        }
        f4(head + i0, u, full + head);
    }
    for (int64_t i = full + threadIdx.x; i < hi; i += kClipThreads) f1(head + i);
}

// The tensor of chunk `c`: the last one whose first chunk is not past it (the first one at least).
template <int N>
__device__ __forceinline__ int tensor_of(const ClipTable<N>& tab, int c) {
    int lo = 0, hi = tab.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (tab.t[mid].first <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// One partial sum of squares per CTA (added to the CTA's own from earlier launches of the call).
// Four 16-byte loads a thread in flight: 2.4 GB in 360 us, 6.7 TB/s, the rate of a copy; 101 MB in
// 24 us (28 with twice the CTAs, in two waves). Loads ahead of the sums, by a ring in shared memory
// or in registers, take 424 to 428 us for 2.4 GB.
template <int N>
__global__ void __launch_bounds__(kClipThreads) clip_norm_kernel(
    const __grid_constant__ ClipTable<N> tab, int add, double* __restrict__ part) {
    __shared__ double red[kClipThreads / 32];
    double acc = 0.0;
    grid_launch_dependents();
    int e = tensor_of(tab, blockIdx.x);
    for (int c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
        while (e + 1 < tab.count && tab.t[e + 1].first <= c) ++e;
        const ClipEntry& E = tab.t[e];
        auto go = [&](auto* g) {
            using S = std::remove_const_t<std::remove_pointer_t<decltype(g)>>;
            walk<S>(
                g, E.n, c - E.first,
                [&](int64_t i) {
                    const double v = to_f(g[i]);
                    acc += v * v;
                },
                [&](int64_t, const uint4(&u)[4], int64_t) { acc += squares<S>(u); });
        };
        if (E.type == MOE_TYPE_BF16) go(static_cast<const __nv_bfloat16*>(E.g));
        else go(static_cast<const float*>(E.g));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kClipThreads / 32; ++i) acc += red[i];
        part[blockIdx.x] = add ? part[blockIdx.x] + acc : acc;
    }
}

// {norm, coef} from the partial sums, in a fixed order; the same value in every CTA.
__device__ __forceinline__ float2 norm_of(const double* __restrict__ part, int nparts, float max_norm) {
    __shared__ double red[kClipThreads / 32];
    __shared__ float2 out;
    grid_dependency_wait();
    double a = 0.0;
    for (int i = threadIdx.x; i < nparts; i += kClipThreads) a += part[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kClipThreads / 32; ++i) a += red[i];
        const float norm = (float)sqrt(a);
        out = make_float2(norm, isfinite(norm) && norm > max_norm ? max_norm / norm : 1.f);
    }
    __syncthreads();
    return out;
}

__global__ void __launch_bounds__(kClipThreads) clip_final_kernel(const double* __restrict__ part,
                                                                  int nparts, float max_norm,
                                                                  float* __restrict__ norm) {
    const float2 r = norm_of(part, nparts, max_norm);
    if (threadIdx.x == 0) {
        norm[0] = r.x;
        norm[1] = r.y;
    }
}

// The factor from the partial sums in every CTA, then the products. 2.4 GB: 750 us, 6.4 TB/s of
// reading and writing with the launch.
template <int N>
__global__ void __launch_bounds__(kClipThreads) clip_scale_kernel(
    const __grid_constant__ ClipTable<N> tab, const double* __restrict__ part, int nparts,
    float max_norm, float* __restrict__ norm) {
    const float2 r = norm_of(part, nparts, max_norm);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        norm[0] = r.x;
        norm[1] = r.y;
    }
    const float coef = r.y;
    // from the last chunk back: the norm's pass left the end of the gradients in L2
    int e = tensor_of(tab, tab.chunks - 1 - blockIdx.x);
    for (int c = tab.chunks - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
        while (tab.t[e].first > c) --e;
        const ClipEntry& E = tab.t[e];
        if (coef == 1.f && E.out == E.g) continue;  // nothing to do in place
        auto go = [&](auto* g) {
            using S = std::remove_const_t<std::remove_pointer_t<decltype(g)>>;
            S* out = static_cast<S*>(E.out);
            const bool vec = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(g)) & 15u) == 0;
            walk<S>(
                g, E.n, c - E.first, [&](int64_t i) { from_f(to_f(g[i]) * coef, out + i); },
                [&](int64_t i0, const uint4(&u)[4], int64_t full) {
                    constexpr int V = Vec<S>::N;
                    const int64_t stride = (int64_t)kClipThreads * V;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int64_t i = i0 + q * stride;
                        if (i >= full) continue;
                        float v[V];
                        Vec<S>::get(u[q], v);
#pragma unroll
                        for (int j = 0; j < V; ++j) v[j] *= coef;
                        if (vec) {
                            __stcs(reinterpret_cast<uint4*>(out + i), Vec<S>::put(v));
                        } else {
#pragma unroll
                            for (int j = 0; j < V; ++j) from_f(v[j], out + i + j);
                        }
                    }
                });
        };
        if (E.type == MOE_TYPE_BF16) go(static_cast<const __nv_bfloat16*>(E.g));
        else go(static_cast<const float*>(E.g));
    }
}

// ------------------------------------------------------------------------------- host side

struct Range {
    uintptr_t lo, hi;
    int tensor;
};

size_t type_bytes(int type) { return type == MOE_TYPE_BF16 ? 2 : 4; }

// The list's own checks: types, sizes, natural alignment, and (with outputs) that no output
// overlaps another tensor's gradient or output: out[i] may only be grads[i] itself.
int check_list(const void* const* g, void* const* out, const int64_t* n, const int* type, int count) {
    for (int i = 0; i < count; ++i) {
        if (type[i] != MOE_TYPE_BF16 && type[i] != MOE_TYPE_F32) return MOE_ERR_INVALID_ARG;
        if (n[i] < 0 || n[i] > ((int64_t)1 << 40)) return MOE_ERR_INVALID_ARG;
        if (n[i] == 0) continue;
        const size_t b = type_bytes(type[i]);
        if (!g[i] || reinterpret_cast<uintptr_t>(g[i]) % b) return MOE_ERR_INVALID_ARG;
        if (out && (!out[i] || reinterpret_cast<uintptr_t>(out[i]) % b)) return MOE_ERR_INVALID_ARG;
    }
    if (!out) return MOE_OK;
    std::vector<Range> r;
    r.reserve(2 * (size_t)count);
    for (int i = 0; i < count; ++i) {
        if (n[i] == 0) continue;
        const uintptr_t bytes = (uintptr_t)n[i] * type_bytes(type[i]);
        const uintptr_t a = reinterpret_cast<uintptr_t>(g[i]), o = reinterpret_cast<uintptr_t>(out[i]);
        r.push_back({o, o + bytes, i});
        if (a != o) r.push_back({a, a + bytes, ~i});
    }
    std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    uintptr_t end_out = 0, end_any = 0;  // ends of the ranges so far: outputs alone, and all
    for (const Range& x : r) {
        const bool is_out = x.tensor >= 0;
        if (x.lo < (is_out ? end_any : end_out)) return MOE_ERR_INVALID_ARG;
        end_any = std::max(end_any, x.hi);
        if (is_out) end_out = std::max(end_out, x.hi);
    }
    return MOE_OK;
}

// Fills a table from tensor `i` on; returns the next tensor.
template <int N>
int fill(ClipTable<N>& tab, const void* const* g, void* const* out, const int64_t* n,
         const int* type, int count, int i) {
    tab.count = 0;
    int64_t chunks = 0;
    for (; i < count && tab.count < N; ++i) {
        if (n[i] == 0) continue;
        const int64_t c = cdiv(n[i], kChunk);
        if (tab.count && chunks + c > INT32_MAX / 2) break;
        tab.t[tab.count++] = {g[i], out ? out[i] : nullptr, n[i], (int32_t)chunks, type[i]};
        chunks += c;
    }
    tab.chunks = (int32_t)chunks;
    return i;
}

// CTAs for a table's chunks, `per_sm` at most: those that an SM holds at once by their registers.
constexpr int kNormCtas = 2, kScaleCtas = 4;
int grid_for(int64_t chunks, int per_sm) {
    int64_t cap = (int64_t)sm_count() * per_sm;
    if (cap > kClipParts) cap = kClipParts;
    return (int)(chunks < 1 ? 1 : chunks < cap ? chunks : cap);
}

template <int N>
int run_clip(const void* const* g, void* const* out, const int64_t* n, const int* type, int count,
             float max_norm, float* norm, double* part, cudaStream_t st) {
    ClipTable<N> tab;
    int nparts = 0, add = 0, launches = 0;
    for (int i = 0; i < count || launches == 0; ++launches) {
        i = fill(tab, g, nullptr, n, type, count, i);
        int grid = grid_for(tab.chunks, kNormCtas);
        if (add && grid > nparts) grid = nparts;  // a later launch adds to the sums of the first
        if (!add) nparts = grid;
        clip_norm_kernel<N><<<grid, kClipThreads, 0, st>>>(tab, add, part);
        if (launch_status() != MOE_OK) return MOE_ERR_LAUNCH;
        add = 1;
    }
    if (!out)
        return launch_dependent(clip_final_kernel, dim3(1), dim3(kClipThreads), 0, st, (const double*)part,
                                nparts, max_norm, norm);
    for (int i = 0, l = 0; i < count || l == 0; ++l) {
        i = fill(tab, g, out, n, type, count, i);
        const int rc = launch_dependent(clip_scale_kernel<N>, dim3(grid_for(tab.chunks, kScaleCtas)),
                                        dim3(kClipThreads), 0, st, tab, (const double*)part, nparts, max_norm, norm);
        if (rc != MOE_OK) return rc;
    }
    return MOE_OK;
}

int clip(const void* const* g, void* const* out, const int64_t* n, const int* type, int count,
         float max_norm, float* norm, void* ws, size_t ws_bytes, moe_stream_t stream) {
    if (!g || !n || !type || !norm || count <= 0) return MOE_ERR_INVALID_ARG;
    if (!(max_norm >= 0.f)) return MOE_ERR_INVALID_ARG;
    int rc = MOE_OK;
    try {
        rc = check_list(g, out, n, type, count);
    } catch (const std::bad_alloc&) {
        return MOE_ERR_TOO_LARGE;
    }
    if (rc != MOE_OK) return rc;
    if (!ws || !aligned16(ws)) return MOE_ERR_WORKSPACE;
    WsCarver wc(ws, ws_bytes);
    double* part = wc.take<double>(kClipParts);
    if (!wc.ok()) return MOE_ERR_WORKSPACE;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    cudaStream_t st = (cudaStream_t)stream;
    return count <= kSmallTable ? run_clip<kSmallTable>(g, out, n, type, count, max_norm, norm, part, st)
                                : run_clip<kLargeTable>(g, out, n, type, count, max_norm, norm, part, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_grad_norm(const void* const* grads, const int64_t* numel, const int* types,
                             int count, float max_norm, float* norm, void* ws, size_t ws_bytes,
                             moe_stream_t stream) {
    return clip(grads, nullptr, numel, types, count, max_norm, norm, ws, ws_bytes, stream);
}

extern "C" int moe_clip_grads(const void* const* grads, void* const* out, const int64_t* numel,
                              const int* types, int count, float max_norm, float* norm, void* ws,
                              size_t ws_bytes, moe_stream_t stream) {
    if (!out) return MOE_ERR_INVALID_ARG;
    return clip(grads, out, numel, types, count, max_norm, norm, ws, ws_bytes, stream);
}
