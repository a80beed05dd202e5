// Choice of experts from router logits, with groups of experts, and its backward.
//
// Per token, with s = sigmoid(l) or softmax(l) over the experts and v = s + b: the E experts
// form n_group groups of E / n_group; a group's score is its largest value or the sum of its
// two largest, the topk_group best groups stay, and the k best experts of those are chosen,
// "larger value, then lower index" throughout. The gate is s of the chosen expert, divided by
// the sum over the chosen ones when asked, times a scale.
//
// The choice is that of the values in 64 bits: two experts' values may lie closer than 32 bits
// tell apart, and which one is chosen should not depend on how a kernel rounds.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "sizes.h"

namespace moe {
namespace {

constexpr int kSelWarps = 8;
constexpr uint32_t kFull = 0xffffffffu;
constexpr int kSiteSelectBwd = 60;

struct SelectParams {
    const float* logits;
    const float* b;
    int64_t T;
    int E, k, mode, n_group, topk_group, rule, renorm;
    float scale;
    int32_t* idx;
    float* gate;
    float* score;
    float* lse;
};

// s = 1 / (1 + e^-l) without overflow on either side.
__device__ __forceinline__ float stable_sigmoid(float l) {
    const float e = expf(-fabsf(l));
    return (l >= 0.f ? 1.f : e) / (1.f + e);  // a NaN takes the second form and stays one
}

// Over the L consecutive lanes that share a token (L a power of two), by a butterfly.
template <int L>
__device__ __forceinline__ float seg_max(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
template <int L, typename F>
__device__ __forceinline__ F seg_sum(F v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
template <int L>
__device__ __forceinline__ int seg_max(int v) {
    if constexpr (L == 32) return __reduce_max_sync(kFull, v);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
template <int L>
__device__ __forceinline__ int seg_min(int v) {
    if constexpr (L == 32) return __reduce_min_sync(kFull, v);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

// Softmax statistics of a row: its largest logit (NaN set aside) and the sum of e^(l - max). A
// row whose logits are all -inf has sum 0.
__device__ __forceinline__ void row_softmax(const float* row, int E, int lane, float& mx, float& sum) {
    mx = -INFINITY;
    for (int e = lane; e < E; e += 32) mx = fmaxf(mx, row[e]);
    mx = seg_max<32>(mx);
    sum = 0.f;
    bool bad = false;
    for (int e = lane; e < E; e += 32) {
        const float l = row[e];
        bad |= l != l;
        if (mx != -INFINITY) sum += expf(l - mx);
    }
    sum = seg_sum<32>(sum);
    if (__any_sync(kFull, bad)) sum = NAN;
}

// Below this sum of the chosen scores one of them may have left fp32's normal range without its
// gate doing so: the gates are then formed in 64 bits.
constexpr float kSmallSum = 9.5367432e-7f;  // 2^-20

// Scores and gates of the chosen experts, stored with the indices: lane `sub` < k of the L lanes
// of a token holds slot `sub`'s expert. `live` masks tokens that are not there, or whose choice
// is made elsewhere. A token whose chosen scores are all zero (in 64 bits) has gates of zero.
// Executed by the whole warp.
template <int L>
__device__ __forceinline__ void finish(const SelectParams& P, int64_t t, int sub, bool live, int my_e,
                                       float mx, float sum) {
    const bool on = live && sub < P.k, sigmoid = P.mode == MOE_MODE_SIGMOID;
    float l = 0.f, s = 0.f;
    if (on) {
        l = P.logits[t * P.E + my_e];
        s = sigmoid ? stable_sigmoid(l) : sum == 0.f ? 0.f : expf(l - mx) / sum;
    }
    float g = s;
    if (P.renorm) {
        const float S = seg_sum<L>(s);
        g = s / S;
        const bool small = S < kSmallSum;
        if (__any_sync(kFull, live && small)) {  // the whole warp: the sum below is collective
            double sd = 0.0;
            if (on && small)
                sd = sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : sum == 0.f ? 0.0 : exp((double)l - (double)mx);
            const double Sd = seg_sum<L>(sd);
            if (small) g = Sd == 0.0 ? 0.f : (float)(sd / Sd);
        }
    }
    if (on) {
        P.idx[t * P.k + sub] = my_e;
        P.gate[t * P.k + sub] = P.scale * g;
        P.score[t * P.k + sub] = s;
    }
    if (live && sub == 0 && !sigmoid && P.lse) P.lse[t] = mx + logf(sum);
}

// Total order of the choice: larger value, then lower index. An index of INT_MAX marks "none".
__device__ __forceinline__ bool before(double v1, int i1, double v2, int i2) {
    if (i1 == INT_MAX || i2 == INT_MAX) return i1 < i2;
    return v1 > v2 || (v1 == v2 && i1 < i2);
}

__device__ __forceinline__ void warp_best(double& v, int& i) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const double ov = __shfl_xor_sync(kFull, v, o);
        const int oi = __shfl_xor_sync(kFull, i, o);
        if (before(ov, oi, v, i)) {
            v = ov;
            i = oi;
        }
    }
}

// The two largest of a warp's values (-inf where there are fewer).
__device__ __forceinline__ void warp_top2(double& a, double& b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const double oa = __shfl_xor_sync(kFull, a, o);
        const double ob = __shfl_xor_sync(kFull, b, o);
        if (oa > a) {
            b = fmax(a, ob);
            a = oa;
        } else {
            b = fmax(b, oa);
        }
    }
}

__device__ __forceinline__ double no_nan(double v) { return v == v ? v : -INFINITY; }

// One token's choice in 64 bits by one warp; lane i < k returns slot i's expert. Any expert
// count up to 256 and any grouping. Lane `lane` holds the experts lane, lane + 32, ...
__device__ int select_exact(const SelectParams& P, int64_t t, int lane, float mx) {
    constexpr int VJ = kMaxExperts / 32;
    const float* row = P.logits + t * P.E;
    const int E = P.E;
    double s[VJ], by[VJ];  // score + bias (a group's sum), and what orders the experts
    double total = 1.0;
    // the scores themselves are needed for values with a bias and for sums over a group
    const bool scores = P.b || (P.n_group > 1 && P.rule == MOE_GROUP_TOP2);
    if (P.mode == MOE_MODE_SOFTMAX && scores) {
        total = 0.0;
#pragma unroll
        for (int j = 0; j < VJ; ++j) {
            const int e = lane + 32 * j;
            s[j] = 0.0;
            if (e < E) {
                const double l = row[e];
                s[j] = mx != -INFINITY ? exp(l - (double)mx) : l == l ? 0.0 : l;
            }
            total += s[j];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
        if (total == 0.0) total = 1.0;  // every logit -inf: scores of zero
    }
#pragma unroll
    for (int j = 0; j < VJ; ++j) {
        const int e = lane + 32 * j;
        by[j] = -INFINITY;
        if (e >= E) continue;
        const double l = row[e];
        if (scores) {
            s[j] = P.mode == MOE_MODE_SOFTMAX ? s[j] / total : 1.0 / (1.0 + exp(-l));
            if (P.b) s[j] += (double)P.b[e];
            s[j] = no_nan(s[j]);
        }
        by[j] = P.b ? s[j] : no_nan(l);  // without a bias the scores have the logits' order
    }
    uint32_t open = 0;  // bit j: expert lane + 32 j can be chosen
#pragma unroll
    for (int j = 0; j < VJ; ++j)
        if (lane + 32 * j < E) open |= 1u << j;
    if (P.n_group > 1) {
        const int per = E / P.n_group;
        double gs = -INFINITY;  // lane g: group g's score
        for (int g = 0; g < P.n_group; ++g) {
            double a = -INFINITY, b = -INFINITY;
#pragma unroll
            for (int j = 0; j < VJ; ++j) {
                const int e = lane + 32 * j;
                if (e < g * per || e >= (g + 1) * per) continue;
                const double v = P.rule == MOE_GROUP_MAX ? by[j] : s[j];
                if (v > a) {
                    b = a;
                    a = v;
                } else {
                    b = fmax(b, v);
                }
            }
            warp_top2(a, b);
            if (lane == g) gs = P.rule == MOE_GROUP_MAX || per == 1 ? a : no_nan(a + b);
        }
        uint32_t kept = 0;  // bit g, the same in every lane
        for (int i = 0; i < P.topk_group; ++i) {
            double v = gs;
            int g = lane < P.n_group && !((kept >> lane) & 1u) ? lane : INT_MAX;
            warp_best(v, g);
            kept |= 1u << g;
        }
#pragma unroll
        for (int j = 0; j < VJ; ++j) {
            const int e = lane + 32 * j;
            if (e < E && !((kept >> (e / per)) & 1u)) open &= ~(1u << j);
        }
    }
    int my_e = 0;
    for (int i = 0; i < P.k; ++i) {
        double v = -INFINITY;
        int e = INT_MAX;
#pragma unroll
        for (int j = 0; j < VJ; ++j)
            if (((open >> j) & 1u) && before(by[j], lane + 32 * j, v, e)) {
                v = by[j];
                e = lane + 32 * j;
            }
        warp_best(v, e);  // k <= the open experts: there is always one
        if ((e & 31) == lane) open &= ~(1u << (e >> 5));
        if (lane == i) my_e = e;
    }
    return my_e;
}

// One token by a whole warp, in 64 bits, with its outputs.
__device__ __noinline__ void select_token(const SelectParams& P, int64_t t, int lane) {
    float mx = 0.f, sum = 1.f;
    if (P.mode == MOE_MODE_SOFTMAX) row_softmax(P.logits + t * P.E, P.E, lane, mx, sum);
    const int my_e = select_exact(P, t, lane, mx);
    finish<32>(P, t, lane, true, my_e, mx, sum);
}

// Every token in 64 bits, one warp each: groupings that the lanes of select_kernel do not hold.
__global__ void __launch_bounds__(kSelWarps * 32) select_exact_kernel(const SelectParams P) {
    const int64_t t = (int64_t)blockIdx.x * kSelWarps + threadIdx.x / 32;
    if (t < P.T) select_token(P, t, threadIdx.x % 32);  // whole warps
}

// ------------------------------------------------------------------- the choice from 32 bits
// L lanes per token (32 / L tokens per warp), each holding up to V consecutive experts of one
// group; lpg lanes (a power of two) hold a group, vr experts each. Every expert becomes one
// integer key, its selection value above its index in the low 8 bits: a lane sorts its keys with
// minima and maxima alone, groups are compared by their lanes' first keys, and each of the k
// rounds takes the largest of the lanes' first keys, which names its expert itself.
//
// The keys are rounded values. Where two of them that the choice has to tell apart lie within
// the rounding's bound, the token is chosen again: the experts that may be among the k are
// evaluated in 64 bits (select_close), or all of them (select_token) where a group's choice is
// in doubt. About one token in 500 takes that way on Gaussian logits.
//
// With a bias the value is s + b in fixed point, 2^-shift units, s by the fast exponential and
// reciprocal; without one it is the logit, whose upper 24 bits order it.
struct SelectLayout {
    int lpg, vr;
    int vec;  // a lane's experts are aligned 16-byte vectors (or none)
};

constexpr float kKeyLimit = 2147483392.f;
constexpr float kU = 5.9604645e-8f;  // 2^-24
// Bounds of the fast scores' errors. Sigmoid: 1 / (1 + e^-l): the quotient is within 2 ulp (4 u
// relative), the sum within u, and the exponential's relative error (1.5 |l| u + 4 u) enters
// times s (1 - s): below 6.4 u in all. Softmax: e^(l - max) / sum: (1.5 |l - max| + 4) u, at
// most 20 u for the sum, its reciprocal and the product; p |l - max| <= 0.37: 25 u p + 0.6 u.
constexpr float kSigmoidErr = 6.4f * kU;
constexpr float kSoftmaxErr = 25.f * kU;

__device__ __forceinline__ int logit_key(float l) {
    const int b = __float_as_int((l == l ? l : -INFINITY) + 0.0f);
    return b ^ ((b >> 31) & 0x7fffffff);
}
// NaN goes to the lower limit.
__device__ __forceinline__ int value_key(float v, float unit) {
    return __float2int_rn(fminf(fmaxf(v * unit, -kKeyLimit), kKeyLimit));
}

template <int V>
__device__ __forceinline__ void sort_desc(int (&k)[V]) {
    auto ce = [&](int a, int b) {
        const int hi = max(k[a], k[b]);
        k[b] = min(k[a], k[b]);
        k[a] = hi;
    };
    if constexpr (V == 2) ce(0, 1);
    if constexpr (V == 4) { ce(0, 1); ce(2, 3); ce(0, 2); ce(1, 3); ce(1, 2); }
    if constexpr (V == 8) {
        ce(0, 1); ce(2, 3); ce(4, 5); ce(6, 7);
        ce(0, 2); ce(1, 3); ce(4, 6); ce(5, 7);
        ce(1, 2); ce(5, 6);
        ce(0, 4); ce(1, 5); ce(2, 6); ce(3, 7);
        ce(2, 4); ce(3, 5);
        ce(1, 2); ce(3, 4); ce(5, 6);
    }
}

// Units of the fixed-point keys for biases of up to `maxb`: |s + b| < 2^(31 - shift).
__device__ __forceinline__ int key_shift(float maxb) {
    return maxb < 1.f ? 30 : maxb < 3.f ? 29 : maxb < 7.f ? 28 : 27;
}

// Score of one expert from its logit, fast (within the bounds above).
__device__ __forceinline__ float fast_score(bool sigmoid, float l, float mx, float inv) {
    return sigmoid ? __fdividef(1.0f, 1.0f + __expf(-l)) : __expf(l - mx) * inv;
}

// One token's choice where its groups are settled (`open`: bit g, group g stays) and the experts
// that may be chosen are those whose key is at least `least`: they are gathered, one per lane,
// evaluated in 64 bits and ranked. More than 32 of them: the token is left to select_token
// (returns false). The keys are formed exactly as select_kernel forms them. Sigmoid scores, or
// logits.
template <bool LOGIT>
__device__ __noinline__ bool select_close(const SelectParams& P, int64_t t, int lane, uint32_t open,
                                          int least, float unit, int* scratch) {
    const float* row = P.logits + t * P.E;
    const int per = P.E / P.n_group;
    int n = 0;
    for (int e0 = 0; e0 < P.E; e0 += 32) {
        const int e = e0 + lane;
        bool in = false;
        if (e < P.E && ((open >> (e / per)) & 1u)) {
            const float l = row[e];
            const int key = LOGIT ? logit_key(l) : value_key(fast_score(true, l, 0.f, 1.f) + P.b[e], unit);
            in = ((key & ~255) | e) >= least;
        }
        const uint32_t m = __ballot_sync(kFull, in);
        const int at = n + __popc(m & ((1u << lane) - 1u));
        if (in && at < 32) scratch[at] = e;
        n += __popc(m);
    }
    if (n > 32) return false;
    __syncwarp();
    int e = INT_MAX;
    double v = 0.0;
    if (lane < n) {
        e = scratch[lane];
        const double l = row[e];
        v = no_nan(LOGIT ? l : 1.0 / (1.0 + exp(-l)) + (double)P.b[e]);
    }
    int rank = 0;
    for (int i = 0; i < n; ++i) {
        const double ov = __shfl_sync(kFull, v, i);
        const int oe = __shfl_sync(kFull, e, i);
        rank += before(ov, oe, v, e) ? 1 : 0;
    }
    __syncwarp();
    if (lane < n && rank < P.k) scratch[rank] = e;
    __syncwarp();
    const int my_e = lane < P.k ? scratch[lane] : 0;
    __syncwarp();
    float mx = 0.f, sum = 1.f;
    if (P.mode == MOE_MODE_SOFTMAX) row_softmax(row, P.E, lane, mx, sum);
    finish<32>(P, t, lane, true, my_e, mx, sum);
    return true;
}

template <int V, int L, bool LOGIT>
__global__ void __launch_bounds__(kSelWarps * 32) select_kernel(const SelectParams P, const SelectLayout Y) {
    constexpr int NT = 32 / L;
    __shared__ int scratch[kSelWarps][32];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = lane % L;
    const int per = P.E / P.n_group, G = P.n_group;
    const bool sigmoid = P.mode == MOE_MODE_SIGMOID;
    const bool top2 = P.rule == MOE_GROUP_TOP2 && per > 1;
    const int g = sub / Y.lpg, r = sub % Y.lpg;
    const int first = g * per + r * Y.vr;
    int count = g < G ? min(Y.vr, per - r * Y.vr) : 0;
    if (count < 0) count = 0;

    float bias[V];
    float unit = 1.f, vmax = 1.f;
    if constexpr (!LOGIT) {
        float mb = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            bias[j] = j < count ? P.b[first + j] : 0.f;
            if (isfinite(bias[j])) mb = fmaxf(mb, fabsf(bias[j]));
        }
        mb = seg_max<L>(mb);
        const int shift = key_shift(mb);
        unit = (float)(1u << shift);
        vmax = (float)(1u << (31 - shift));
    }

    const int64_t stride = (int64_t)gridDim.x * kSelWarps * NT;
    for (int64_t t0 = ((int64_t)blockIdx.x * kSelWarps + warp) * NT; t0 < P.T; t0 += stride) {
        const int64_t t = t0 + lane / L;
        const bool live = t < P.T;
        float l[V];
#pragma unroll
        for (int j = 0; j < V; ++j) l[j] = 0.f;
        if (live) {
            const float* src = P.logits + t * P.E + first;
            if (V >= 4 && Y.vec) {
                if (count == V) {
#pragma unroll
                    for (int j = 0; j + 3 < V; j += 4) {
                        const float4 a = *reinterpret_cast<const float4*>(src + j);
                        l[j] = a.x, l[(j + 1) % V] = a.y, l[(j + 2) % V] = a.z, l[(j + 3) % V] = a.w;
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (j < count) l[j] = src[j];
            }
        }
        bool odd = false;  // not a row for this kernel's arithmetic
        float mx = 0.f, sum = 1.f, inv = 1.f;
        if (!sigmoid) {
            mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < count) mx = fmaxf(mx, l[j]);
            mx = seg_max<L>(mx);
            sum = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < count) sum += __expf(l[j] - mx);
            sum = seg_sum<L>(sum);
            odd = !(sum < 1e30f) || mx == -INFINITY;  // NaN or infinite logits
            inv = __fdividef(1.0f, sum);
        }
        int key[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int k = LOGIT ? logit_key(l[j]) : value_key(fast_score(sigmoid, l[j], mx, inv) + bias[j], unit);
            key[j] = j < count ? (k & ~255) | (first + j) : INT_MIN;
        }
        // how far apart two keys have to be to settle their order: twice the value's error (the
        // score's, the sum's rounding and the fixed point's), and the index bits
        int tol = 0;
        if constexpr (!LOGIT) {
            const float es = sigmoid ? kSigmoidErr : kSoftmaxErr * inv + 0.6f * kU;
            tol = 260 + (int)ceilf(2.f * (es + kU * vmax) * unit);
        }
        uint32_t open = 1u;
        int gs = 0;
        float fa = -INFINITY, fb = -INFINITY;
        if (LOGIT && top2 && G > 1) {  // a lane's two largest logits
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float x = j < count && l[j] == l[j] ? l[j] : -INFINITY;
                fb = fmaxf(fb, fminf(fa, x));
                fa = fmaxf(fa, x);
                odd |= j < count && l[j] != l[j];  // a NaN's score counts as -inf in the sum
            }
        }
        sort_desc<V>(key);
        if (G > 1) {
            int a = key[0], b = V > 1 ? key[1 % V] : INT_MIN;
            for (int o = 1; o < Y.lpg; o <<= 1) {
                if (LOGIT && top2) {
                    const float oa = __shfl_xor_sync(kFull, fa, o), ob = __shfl_xor_sync(kFull, fb, o);
                    fb = fmaxf(fmaxf(fb, ob), fminf(fa, oa));
                    fa = fmaxf(fa, oa);
                } else {
                    const int oa = __shfl_xor_sync(kFull, a, o), ob = __shfl_xor_sync(kFull, b, o);
                    b = max(max(b, ob), min(a, oa));
                    a = max(a, oa);
                }
            }
            if (!top2) gs = a;
            else if (!LOGIT) gs = (a >> 1) + (b >> 1);
            else gs = __float_as_int(fast_score(sigmoid, fa, mx, inv) + fast_score(sigmoid, fb, mx, inv));
            // a sum with a value beyond the keys' range, or a second value that does not count
            if (!LOGIT && top2 && g < G) odd |= b <= -(int)kKeyLimit + 512 || a >= (int)kKeyLimit - 512;
            int rank = 0;
            for (int h = 0; h < G; ++h) {
                const int x = __shfl_sync(kFull, gs, h * Y.lpg, L);
                rank += x > gs || (x == gs && h < g);
            }
            const bool kept = g < G && rank < P.topk_group;
            if (P.topk_group < G) {
                const int lo = seg_min<L>(kept ? gs : INT_MAX);
                const int hi = seg_max<L>(!kept && g < G ? gs : INT_MIN);
                if (LOGIT && top2) {  // sums of scores: softmax terms are within 160 u of themselves
                    const float x = __int_as_float(lo), y = __int_as_float(hi);  // down to e^-87
                    odd |= !(x - y > 2.f * (sigmoid ? 2.f * kSigmoidErr + kU * x : 161.f * kU * x)) || x < 1e-30f;
                } else if (LOGIT) {
                    odd |= (lo >> 8) == (hi >> 8);
                } else {
                    odd |= (uint32_t)lo - (uint32_t)hi <= (uint32_t)tol;
                }
            }
            const uint32_t bits = __ballot_sync(kFull, kept && r == 0);
            open = 0u;
            for (int h = 0; h < G; ++h) open |= ((bits >> (lane / L * L + h * Y.lpg)) & 1u) << h;
            if (!kept) {
#pragma unroll
                for (int j = 0; j < V; ++j) key[j] = INT_MIN;
            }
        }
        int my_key = 0, prev = 0;
        bool close = false;
        for (int i = 0; i <= P.k; ++i) {
            const int w = seg_max<L>(key[0]);
            if (i > 0) close |= LOGIT ? (w >> 8) == (prev >> 8) : (uint32_t)prev - (uint32_t)w <= (uint32_t)tol;
            if (i == 0 && !LOGIT) odd |= w >= (int)kKeyLimit - 512;
            if (i == P.k) break;
            prev = w;
            if (sub == i) my_key = w;
            if (key[0] == w) {
#pragma unroll
                for (int j = 0; j + 1 < V; ++j) key[j] = key[j + 1];
                key[V - 1] = INT_MIN;
            }
        }
        // prev is the k-th key: what is not below it by more than the bound may be chosen
        const uint32_t flagged = __ballot_sync(kFull, live && (odd || close));
        const uint32_t oddball = __ballot_sync(kFull, live && odd);
        const uint32_t mask = L == 32 ? kFull : ((1u << (L % 32)) - 1u) << (lane / L * L);
        finish<L>(P, t, sub, live && !(flagged & mask), my_key & 255, mx, sum);
        if (flagged) {
            for (int q = 0; q < NT; ++q) {  // the warp together, one token at a time
                const uint32_t m = L == 32 ? kFull : ((1u << (L % 32)) - 1u) << (q * L);
                if (!(flagged & m)) continue;
                const int least = __shfl_sync(kFull, prev, q * L);
                const uint32_t o = __shfl_sync(kFull, open, q * L);
                const int by = LOGIT ? 255 : __shfl_sync(kFull, tol, q * L);
                const bool all = (oddball & m) || (!LOGIT && !sigmoid);
                const int from = LOGIT ? least & ~255 : least < INT_MIN + by ? INT_MIN : least - by;
                if (all || !select_close<LOGIT>(P, t0 + q, lane, o, from, unit, scratch[warp]))
                    select_token(P, t0 + q, lane);
            }
        }
    }
}

// ---------------------------------------------------------------------------- backward
// ds_i = scale / S (dg_i - sum_j (s_j / S) dg_j) with renormalised gates (0 where S is 0), else
// scale dg_i. Sigmoid: dl = ds_i s_i (1 - s_i) on the chosen experts. Softmax: dl_e = p_e
// (ds_e - sum_i s_i ds_i), ds_e zero off the chosen experts; with renormalised gates that sum
// is zero, so only the chosen experts have a gradient. z-loss: + (2 z_coef / T) lse p_e.
//
// Bound by writing dlogits. L lanes hold a token's slots (L >= k), so a warp forms the gradients of
// 32 / L tokens at once; it scatters them into zeroed rows in shared memory and stores the rows
// whole, since the tokens' rows are one piece of memory.
struct SelectBwdParams {
    const float* dg;
    const int32_t* idx;
    const float* score;
    const float* logits;
    const float* lse;
    const float* extra;
    int64_t T;
    int E, k, mode, renorm;
    float scale, z_scale;
    float* dlogits;
    int* status;
};

template <int L>
__global__ void __launch_bounds__(kSelWarps * 32) select_bwd_kernel(const SelectBwdParams P) {
    constexpr int NT = 32 / L;
    extern __shared__ __align__(16) float rows[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = lane % L;
    const int E = P.E, k = P.k;
    // one warp's rows; a multiple of 16 bytes
    float* row = rows + (size_t)warp * ((NT * E + 3) / 4 * 4);
    const int64_t t0 = ((int64_t)blockIdx.x * kSelWarps + warp) * NT;
    if (t0 >= P.T) return;  // whole warp
    const int64_t t = t0 + lane / L;
    const int n = (int)min((int64_t)NT, P.T - t0) * E;  // elements of the warp's tokens
    const bool softmax = P.mode == MOE_MODE_SOFTMAX;
    const bool dense = softmax && (!P.renorm || P.z_scale != 0.f);
    for (int i = 4 * lane; i < n; i += 128)
        *reinterpret_cast<float4*>(row + i) = make_float4(0.f, 0.f, 0.f, 0.f);
    int e = -1;
    float s = 0.f, dg = 0.f;
    if (t < P.T && sub < k) {
        e = P.idx[t * k + sub];
        if (e < 0 || e >= E) {  // the slot is dropped
            record_error(P.status, MOE_ERR_BAD_INDEX, kSiteSelectBwd);
            e = -1;
        } else {
            s = P.score[t * k + sub];
            dg = P.dg[t * k + sub];
        }
    }
    float ds = P.scale * dg;
    if (P.renorm) {
        const float S = seg_sum<L>(s);
        const float m = seg_sum<L>(s / S * dg);
        ds = S == 0.f ? 0.f : P.scale / S * (dg - m);
    }
    float c = 0.f;
    if (softmax && !P.renorm) c = seg_sum<L>(s * ds);
    float v = dense ? ds : softmax ? ds * s : ds * s * (1.f - s);
    // an expert named twice in a token gets its slots' terms summed in slot order, by the first
    const uint32_t same = __match_any_sync(kFull, e < 0 ? -1 - lane : lane / L * E + e);
    if (__any_sync(kFull, (same & (same - 1)) != 0)) {
        float sum = 0.f;
        for (int i = 0; i < 32; ++i) {
            const float o = __shfl_sync(kFull, v, i);
            if ((same >> i) & 1u) sum += o;
        }
        v = sum;
        if ((same & ((1u << lane) - 1u)) != 0) e = -1;
    }
    __syncwarp();
    if (e >= 0) row[lane / L * E + e] = v;
    __syncwarp();
    float* out = P.dlogits + t0 * E;
    const float* extra = P.extra ? P.extra + t0 * E : nullptr;
    if (dense) {
        const float* l = P.logits + t0 * E;
        for (int q = 0; q * E < n; ++q) {
            const float l_se = P.lse[t0 + q];
            const float cq = __shfl_sync(kFull, c, q * L);
            const float zl = P.z_scale * l_se;
            for (int i = q * E + lane; i < (q + 1) * E; i += 32) {
                float g = 0.f;
                if (l_se != -INFINITY) {  // else no expert has a score
                    const float p = expf(l[i] - l_se);
                    g = p * (row[i] - cq) + zl * p;
                }
                out[i] = extra ? g + extra[i] : g;
            }
        }
        return;
    }
    const bool vec = ((reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(extra)) & 15u) == 0;
    const int nv = vec ? n / 4 * 4 : 0;
    for (int i = 4 * lane; i < nv; i += 128) {
        float4 g = *reinterpret_cast<const float4*>(row + i);
        if (extra) {
            const float4 x = *reinterpret_cast<const float4*>(extra + i);
            g.x += x.x, g.y += x.y, g.z += x.z, g.w += x.w;
        }
        *reinterpret_cast<float4*>(out + i) = g;
    }
    for (int i = nv + lane; i < n; i += 32) out[i] = extra ? row[i] + extra[i] : row[i];
}

template <int L>
int launch_lanes(const SelectParams& P, const SelectLayout& Y, cudaStream_t st) {
    constexpr int NT = 32 / L;
    int64_t blocks = cdiv(P.T, (int64_t)kSelWarps * NT);
    const int64_t cap = (int64_t)sm_count() * 4;
    if (blocks > cap) blocks = cap;
    auto go = [&](auto kern) { kern<<<(unsigned)blocks, kSelWarps * 32, 0, st>>>(P, Y); };
    auto pick = [&](auto logit) {
        constexpr bool LOGIT = decltype(logit)::value;
        if (Y.vr <= 1) go(select_kernel<1, L, LOGIT>);
        else if (Y.vr <= 2) go(select_kernel<2, L, LOGIT>);
        else if (Y.vr <= 4) go(select_kernel<4, L, LOGIT>);
        else go(select_kernel<8, L, LOGIT>);
    };
    if (P.b) pick(std::false_type());
    else pick(std::true_type());
    return launch_status();
}

// The lanes of a token: the fewest per group (a power of two) that hold its experts at 8 each, and
// at least one per slot. Groupings that need more than 32 lanes (their number no power of two
// and their experts too many) are chosen in 64 bits throughout.
int launch_select(const SelectParams& P, cudaStream_t st) {
    const int per = P.E / P.n_group;
    SelectLayout Y{1, 0, 0};
    while (Y.lpg * 8 < per) Y.lpg *= 2;
    int L = 8;
    while (L < P.n_group * Y.lpg || L < P.k) L *= 2;
    if (L > 32) {
        select_exact_kernel<<<(unsigned)cdiv(P.T, kSelWarps), kSelWarps * 32, 0, st>>>(P);
        return launch_status();
    }
    while (P.n_group * Y.lpg * 2 <= L && Y.lpg < per) Y.lpg *= 2;  // no lanes left over
    Y.vr = (int)cdiv(per, Y.lpg);
    Y.vec = (Y.vr == 8 || Y.vr == 4) && per % Y.vr == 0 && aligned16(P.logits);
    return L == 8 ? launch_lanes<8>(P, Y, st) : L == 16 ? launch_lanes<16>(P, Y, st) : launch_lanes<32>(P, Y, st);
}

template <int L>
int launch_bwd_lanes(const SelectBwdParams& P, cudaStream_t st) {
    constexpr int NT = 32 / L;
    const size_t smem = sizeof(float) * kSelWarps * ((NT * P.E + 3) / 4 * 4);  // 32 KB at most
    select_bwd_kernel<L><<<(unsigned)cdiv(P.T, (int64_t)kSelWarps * NT), kSelWarps * 32, smem, st>>>(P);
    return launch_status();
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_select_experts(const float* logits, const float* b, int64_t T, int E, int k,
                                  int mode, int n_group, int topk_group, int group_rule, int renorm,
                                  float scale, int32_t* topk_idx, float* topk_gate,
                                  float* topk_score, float* lse, moe_stream_t stream) {
    if (!logits || !topk_idx || !topk_gate || !topk_score) return MOE_ERR_INVALID_ARG;
    if (T <= 0 || E <= 0 || k <= 0 || n_group <= 0 || topk_group <= 0) return MOE_ERR_INVALID_ARG;
    if (mode != MOE_MODE_SIGMOID && mode != MOE_MODE_SOFTMAX) return MOE_ERR_INVALID_ARG;
    if (group_rule != MOE_GROUP_MAX && group_rule != MOE_GROUP_TOP2) return MOE_ERR_INVALID_ARG;
    if (topk_group > n_group || E % n_group != 0) return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts || k > E || k > 32 || n_group > kMaxGroups) return MOE_ERR_UNSUPPORTED;
    if (k > topk_group * (E / n_group)) return MOE_ERR_INVALID_ARG;
    if (cdiv(T, kSelWarps) > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    const SelectParams P{logits, b, T, E, k, mode, n_group, topk_group, group_rule, renorm ? 1 : 0,
                         scale, topk_idx, topk_gate, topk_score, lse};
    return launch_select(P, (cudaStream_t)stream);
}

extern "C" int moe_select_experts_bwd(const float* dg, const int32_t* topk_idx,
                                      const float* topk_score, const float* logits,
                                      const float* lse, const float* dlogits_extra, int64_t T,
                                      int E, int k, int mode, int renorm, float scale, float z_coef,
                                      float* dlogits, moe_stream_t stream) {
    if (!dg || !topk_idx || !topk_score || !dlogits) return MOE_ERR_INVALID_ARG;
    if (T <= 0 || E <= 0 || k <= 0) return MOE_ERR_INVALID_ARG;
    if (mode != MOE_MODE_SIGMOID && mode != MOE_MODE_SOFTMAX) return MOE_ERR_INVALID_ARG;
    if (z_coef != 0.f && mode != MOE_MODE_SOFTMAX) return MOE_ERR_INVALID_ARG;
    const bool dense = mode == MOE_MODE_SOFTMAX && (!renorm || z_coef != 0.f);
    if (dense && (!logits || !lse)) return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts || k > E || k > 32) return MOE_ERR_UNSUPPORTED;
    if (cdiv(T, kSelWarps) > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    int* status = device_status_word();
    if (!status) return MOE_ERR_LAUNCH;
    const SelectBwdParams P{dg, topk_idx, topk_score, logits, lse, dlogits_extra, T, E, k, mode,
                            renorm ? 1 : 0, scale, 2.0f * z_coef / (float)T, dlogits, status};
    cudaStream_t st = (cudaStream_t)stream;
    return k <= 8 ? launch_bwd_lanes<8>(P, st) : k <= 16 ? launch_bwd_lanes<16>(P, st) : launch_bwd_lanes<32>(P, st);
}
