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

#include "common.cuh"
#include "select_key.h"
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

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// x / y for y within [2^-20, 2^20] by one correction of the quotient with its exact remainder
// (Markstein): within one unit in the last place, without a division's slow path.
__device__ __forceinline__ float quotient(float x, float y) {
    const float r = fast_rcp(y);
    const float q = x * r;
    return fmaf(fmaf(-q, y, x), r, q);
}

// s = 1 / (1 + e^-l) without overflow on either side.
__device__ __forceinline__ float stable_sigmoid(float l) {
    const float e = expf(-fabsf(l));
    return quotient(l >= 0.f ? 1.f : e, 1.f + e);  // a NaN takes the second form and stays one
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
    if constexpr (L == 32) {
        return __reduce_max_sync(kFull, v);
    } else {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
        return v;
    }
}
template <int L>
__device__ __forceinline__ int seg_min(int v) {
    if constexpr (L == 32) {
        return __reduce_min_sync(kFull, v);
    } else {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(kFull, v, o));
        return v;
    }
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
// of a token holds slot `sub`'s expert and that expert's logit. `live` masks tokens that are not
// there, or whose choice is made elsewhere. A token whose chosen scores are all zero (in 64 bits)
// has gates of zero. Executed by the whole warp.
template <int L>
__device__ __forceinline__ void finish(const SelectParams& P, int64_t t, int sub, bool live, int my_e,
                                       float l, float mx, float sum) {
    const bool on = live && sub < P.k, sigmoid = P.mode == MOE_MODE_SIGMOID;
    float s = 0.f;
    if (on) s = sigmoid ? stable_sigmoid(l) : sum == 0.f ? 0.f : expf(l - mx) / sum;
    float g = s;
    if (P.renorm) {
        const float S = seg_sum<L>(s);
        g = quotient(s, S);
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

// The same for one token by a whole warp, in the paths that are taken seldom.
__device__ __noinline__ void finish_token(const SelectParams& P, int64_t t, int lane, int my_e, float l, float mx,
                                          float sum) {
    finish<32>(P, t, lane, true, my_e, l, mx, sum);
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

// A score in 64 bits; total: the softmax's sum. One copy of the code, which runs seldom and cold.
__device__ __noinline__ double score64(bool sigmoid, float l, float mx, double total) {
    const double e = exp(sigmoid ? -(double)l : (double)l - (double)mx);
    return (sigmoid ? 1.0 : e) / (sigmoid ? 1.0 + e : total);
}

// Integers in the order of 64-bit values (of which none is NaN); -0 and 0 are one.
__device__ __forceinline__ long long order_of(double v) {
    const long long b = __double_as_longlong(v + 0.0);
    return b ^ ((b >> 63) & 0x7fffffffffffffffll);
}
__device__ __forceinline__ bool ahead_of(long long v1, int i1, long long v2, int i2) {
    return v1 > v2 || (v1 == v2 && i1 < i2);
}

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
    finish_token(P, t, lane, my_e, lane < P.k ? P.logits[t * P.E + my_e] : 0.f, mx, sum);
}

// ------------------------------------------------------------------- the choice from 32 bits
// L lanes per token (32 / L tokens per warp), each holding up to 8 NB consecutive experts of one
// group; lpg lanes (a power of two) hold a group, vr experts each. A warp copies its next tokens'
// logits to shared memory while it works on the present ones. Every expert becomes one integer
// key: its selection value as a 23-bit fixed-point number above its index. A lane sorts its keys
// by minima and maxima alone and keeps the eight largest, groups are compared by their lanes'
// first keys, and the k largest of the lanes' sorted keys come from a merge across eight lanes
// that halves what a lane holds at each step (or, for more lanes, from k rounds that take the
// largest of the lanes' first keys).
//
// The keys are rounded values. Where two that the choice has to tell apart lie within the
// rounding's bound, the warp evaluates those near the border in 64 bits, one token at a time, and
// ranks them: groups in settle_groups, the slots' experts in settle_slots. Rows that are not for
// this arithmetic (NaN, infinities, more than 32 experts near the border) are chosen in 64 bits
// throughout.
//
// Bound by latency and occupancy: 65,536 tokens of 256 experts in 8 groups take 31 to 32 us (1190
// instructions and 4.4 us per step of four tokens and warp, 54% of the issue slots with the 16 warps
// per SM that 128 registers leave; several of the kernels spill 32 to 108 bytes at that), 29 us where
// no token comes near a border, 10.8 us for their bytes. 16,383 tokens of 160, softmax: 11.1 us, 9.5 without
// near ties. Rows that are no whole vectors a lane cost little more: 65,536 tokens of 40 experts in one
// group 16.3 us, 72 19.5, 100 21.5 (64 and 128, in vectors: 15.7 and 20.4). A token near a border took 6 to
// 11 us of latency when its choice was made anew, nearly all of it instructions that the SM has not met
// before (a 64-bit one also takes 64 cycles a warp): so what the keys have settled is kept, loops
// over its few candidates stay rolled, and the 64-bit score is one piece of code.
//
// What is slow: tokens that are chosen in 64 bits throughout. With biases that are all equal a token
// of equal logits (padding) is one; one such token in 64 makes the large case 98 us, 53 with biases of 41
// levels. A bias of +inf, or a whole group's biases 16 or more below the largest, sends every token
// there: 2.1 to 2.2 ms. Without a bias a whole group's logits 16 or more below the largest has every
// token's groups settled from its logits: 0.43 ms. (Single experts masked by -inf, in logits or biases,
// and with a bias a whole group's logits, cost nothing.)
//
// With a bias the value is s + (b - base), base the smallest bias within 16 of the largest, s by
// the fast exponential and reciprocal, scaled so that it lies below 1 and clamped at 0. Without
// one it is the logit, from 16 below the row's largest up.
struct SelectLayout {
    int lpg, vr;
};

constexpr float kU = 5.9604645e-8f;  // 2^-24
// Bounds of the fast scores' errors. Sigmoid: 1 / (1 + e^-l): the reciprocal is within 1 ulp (2 u
// relative), the sum within u, and the exponential's relative error (1.5 |l| u + 4 u) enters
// times s (1 - s): below 5 u in all; 6.4 u leaves room. Softmax: p = e^(l - max) / sum, where 1 / sum
// is the row's largest p, P. A term is off by (2.3 |l - max| + 4) u of itself (the roundings of the
// difference, of log2 e and of their product), and p |l - max| <= 0.37 P: 10 u P for two values. The sum
// is off by 4 u, 2.3 u times the mean of |l - max| over p (at most ln 256, as the entropy is) and 13
// roundings, its reciprocal and their products by 4 u: 34 u, a factor that the row's values have in
// common, so it moves the difference of two by 34 u P at most. Twice the bound, 50 u P + 1.2 u, covers both.
constexpr float kSigmoidErr = 6.4f * kU;
constexpr float kSoftmaxErr = 25.f * kU;
constexpr float kLog2e = 1.44269504f;

// Score of one expert from its logit (within the bounds above); inv = 1 / sum for softmax.
__device__ __forceinline__ float fast_score(bool sigmoid, float l, float mx, float inv) {
    return sigmoid ? fast_rcp(1.0f + fast_exp2(-kLog2e * l)) : fast_exp2(kLog2e * (l - mx)) * inv;
}
__device__ __forceinline__ float score_err(bool sigmoid, float inv) {
    return sigmoid ? kSigmoidErr : kSoftmaxErr * inv + 0.6f * kU;
}
__device__ __forceinline__ int logit_key(float l) {
    const int b = __float_as_int((l == l ? l : -INFINITY) + 0.0f);
    return b ^ ((b >> 31) & 0x7fffffff);
}

// The key of a value v = a x + b clamped to [0, 1) (a NaN to 0), rounded to half a unit.
__device__ __forceinline__ int fixed_key(float x, float a, float b, int id) {
    float v;
    asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(v) : "f"(x), "f"(a), "f"(b));
    return key_of(__float_as_uint(v + 1.0f), id);
}
constexpr float kLogitRange = 16.f;
constexpr float kBelowOne = 0.9990234f;  // 1 - 2^-10

// The biases' base, the smallest within 16 of the largest finite one (0 where none is finite), and
// 1 + the largest's distance from it; from a warp's b[j] = bias of expert lane + 32 j (NaN past
// the last). An infinite bias gives an infinite range.
__device__ __forceinline__ float bias_base(const float (&b)[kMaxExperts / 32], float& range) {
    float hi = -INFINITY;
    bool inf = false;
#pragma unroll
    for (int j = 0; j < kMaxExperts / 32; ++j) {
        if (isfinite(b[j])) hi = fmaxf(hi, b[j]);
        inf |= b[j] == INFINITY;
    }
    hi = seg_max<32>(hi);
    float lo = INFINITY;
#pragma unroll
    for (int j = 0; j < kMaxExperts / 32; ++j)
        if (b[j] >= hi - 16.f && b[j] <= hi) lo = fminf(lo, b[j]);
    lo = -seg_max<32>(-lo);
    if (!isfinite(lo)) lo = hi = 0.f;
    range = __any_sync(kFull, inf) ? INFINITY : 1.f + (hi - lo);
    return lo;
}

// The sum of e^(l - max) over a row in shared memory, in 64 bits.
__device__ __noinline__ double softmax_total(const float* row, int E, int lane, float mx) {
    double total = 0.0;
#pragma unroll 1
    for (int e = lane; e < E; e += 32) total += exp((double)row[e] - (double)mx);
    return seg_sum<32>(total);
}

// Which groups of a token stay, where its keys leave that open, by a whole warp: lane g finds group
// g's largest keys among the first four of the lanes that hold it (`keys`: eight per lane), those
// that may be its two largest are evaluated in 64 bits, and the groups are ranked. False where
// three candidates a group are not enough.
__device__ __noinline__ bool settle_groups(const SelectParams& P, int lane, const float* row, const int* keys,
                                           int lpg, int tol, float mx, uint32_t& open) {
    const int G = P.n_group, per = P.E / G;
    const bool sigmoid = P.mode == MOE_MODE_SIGMOID, top2 = P.rule == MOE_GROUP_TOP2 && per > 1;
    int a = INT_MIN, b = INT_MIN, c = INT_MIN, d = INT_MIN;
    if (lane < G) {
#pragma unroll 1
        for (int h = 0; h < lpg; ++h) {
            const int4 u = *reinterpret_cast<const int4*>(keys + (lane * lpg + h) * 8);
            const int v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int x = min(a, v[q]), y = min(b, x), z = min(c, y);
                a = max(a, v[q]);
                b = max(b, x);
                c = max(c, y);
                d = max(d, z);
            }
        }
    }
    // the two largest (or the largest) are among the first three unless the fourth may reach them
    if (__any_sync(kFull, lane < G && per > 3 && units_of(top2 ? b : a) - units_of(d) <= tol)) return false;
    const double total = sigmoid ? 1.0 : softmax_total(row, P.E, lane, mx);
    // three candidates a group, all of them at once where there are lanes for that
    double v[3] = {-INFINITY, -INFINITY, -INFINITY};
    const int step = 3 * G <= 32 ? 3 : 1, h = lane % G, q = lane / G;
#pragma unroll 1
    for (int i = 0; i < 3; i += step) {
        const int ka = __shfl_sync(kFull, a, h), kb = __shfl_sync(kFull, b, h), kc = __shfl_sync(kFull, c, h);
        const int which = step == 3 ? q : i, k = which == 0 ? ka : which == 1 ? kb : which == 2 ? kc : INT_MIN;
        double x = -INFINITY;
        if (k != INT_MIN) x = no_nan(score64(sigmoid, row[expert_of(k)], mx, total) + (double)P.b[expert_of(k)]);
        if (step == 3) {
#pragma unroll
            for (int r = 0; r < 3; ++r) v[r] = __shfl_sync(kFull, x, h + r * G);
        } else {
            v[0] = i == 0 ? x : v[0];
            v[1] = i == 1 ? x : v[1];
            v[2] = i == 2 ? x : v[2];
        }
    }
    double gs = -INFINITY;
    if (lane < G) {
        const double x = fmax(v[0], v[1]), y = fmin(v[0], v[1]);
        gs = top2 ? no_nan(fmax(x, v[2]) + fmax(y, fmin(x, v[2]))) : fmax(x, v[2]);
    }
    int rank = 0;
    const long long mine = order_of(gs);
    for (int g = 0; g < G; ++g) rank += ahead_of(__shfl_sync(kFull, mine, g), g, mine, lane);
    open = __ballot_sync(kFull, lane < G && rank < P.topk_group);
    return true;
}

// Which experts a token's slots hold, where the keys leave their order or the last one open, by a
// whole warp: those of its lanes' keys that may be among the k largest are gathered, one per lane,
// evaluated (without a bias: the logits themselves) and ranked; list[i] = slot i's expert. False where
// they are more than 32.
template <bool LOGIT>
__device__ __noinline__ bool settle_slots(const SelectParams& P, int lane, const float* row, const int* keys,
                                          int nkeys, int least, float mx, int* list) {
    const bool sigmoid = P.mode == MOE_MODE_SIGMOID;
    int n = 0;
#pragma unroll 1
    for (int c = lane; c < nkeys; c += 32) {
        const int key = keys[c];
        const bool in = key != INT_MIN && units_of(key) >= least;
        const uint32_t m = __ballot_sync(kFull, in);
        const int at = n + __popc(m & ((1u << lane) - 1u));
        if (in && at < 32) list[at] = expert_of(key);
        n += __popc(m);
    }
    if (n > 32 || n < P.k) return false;
    const double total = LOGIT || sigmoid ? 1.0 : softmax_total(row, P.E, lane, mx);
    __syncwarp();
    int e = INT_MAX;
    long long x = 0;
    if (lane < n) {
        e = list[lane];
        if (LOGIT) x = logit_key(row[e]);
        else x = order_of(no_nan(score64(sigmoid, row[e], mx, total) + (double)P.b[e]));
    }
    int rank = 0;
    for (int i = 0; i < n; ++i) rank += ahead_of(__shfl_sync(kFull, x, i), __shfl_sync(kFull, e, i), x, e);
    __syncwarp();
    if (lane < n && rank < P.k) list[rank] = e;
    __syncwarp();
    return true;
}

// One token without a bias whose groups, or more logits than its lanes list, the keys leave open, by
// a whole warp, from its logits in shared memory: groups by their largest logits or (in 64 bits)
// the scores of the two largest, then k times the largest logit left.
__device__ __noinline__ void select_logits(const SelectParams& P, int64_t t, int lane, const float* row) {
    constexpr int VJ = kMaxExperts / 32;
    const int E = P.E, G = P.n_group, per = E / G, k = P.k;
    const bool sigmoid = P.mode == MOE_MODE_SIGMOID, top2 = P.rule == MOE_GROUP_TOP2 && per > 1;
    float l[VJ];  // of the experts lane, lane + 32, ...
#pragma unroll
    for (int j = 0; j < VJ; ++j) l[j] = lane + 32 * j < E ? row[lane + 32 * j] : -INFINITY;
    float mx = 0.f, sum = 1.f;
    if (!sigmoid) {
        mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < VJ; ++j) mx = fmaxf(mx, l[j]);
        mx = seg_max<32>(mx);
        sum = 0.f;
#pragma unroll
        for (int j = 0; j < VJ; ++j) sum += fast_exp2(kLog2e * (l[j] - mx));
        sum = seg_sum<32>(sum);
    }
    bool same = true;  // all logits: a padded token's
#pragma unroll
    for (int j = 0; j < VJ; ++j) same &= lane + 32 * j >= E || l[j] == row[0];
    if (__all_sync(kFull, same)) {  // the first experts of the first groups
        finish_token(P, t, lane, lane < k ? lane : 0, row[0], mx, sum);
        return;
    }
    uint32_t open = 1u;
    if (G > 1) {
        int a = INT_MIN, b = INT_MIN, ia = 0, ib = 0;  // lane g: group g's two largest
        if (lane < G) {
#pragma unroll 4
            for (int e = lane * per; e < (lane + 1) * per; ++e) {
                const int v = logit_key(row[e]);
                const bool A = v > a, B = v > b;
                b = A ? a : B ? v : b;
                ib = A ? ia : B ? e : ib;
                a = A ? v : a;
                ia = A ? e : ia;
            }
        }
        double gs = -INFINITY;  // (a common factor, the softmax's sum, leaves the order)
        if (lane < G)
            gs = top2 ? score64(sigmoid, row[ia], mx, 1.0) + score64(sigmoid, row[ib], mx, 1.0)
                      : no_nan((double)row[ia]);
        int rank = 0;
        const long long mine = order_of(gs);
        for (int h = 0; h < G; ++h) rank += ahead_of(__shfl_sync(kFull, mine, h), h, mine, lane);
        open = __ballot_sync(kFull, lane < G && rank < P.topk_group);
    }
    int key[VJ];  // INT_MIN, below every value, past the last expert and in closed groups
#pragma unroll
    for (int j = 0; j < VJ; ++j) {
        const int e = lane + 32 * j;
        key[j] = e < E && ((open >> (e / per)) & 1u) ? logit_key(l[j]) : INT_MIN;
    }
    int my_e = 0;
    uint32_t taken = 0;
    for (int i = 0; i < k; ++i) {  // the largest key left, of the lowest index
        int best = INT_MIN, e = INT_MAX;
#pragma unroll
        for (int j = 0; j < VJ; ++j)
            if (!((taken >> j) & 1u) && key[j] > best) {
                best = key[j];
                e = lane + 32 * j;
            }
        const int top = __reduce_max_sync(kFull, best);
        const int w = __reduce_min_sync(kFull, best == top ? e : INT_MAX);
        if ((w & 31) == lane) taken |= 1u << (w >> 5);
        if (lane == i) my_e = w;
    }
    finish_token(P, t, lane, my_e, lane < k ? row[my_e] : 0.f, mx, sum);
}

// Sorting network for eight keys, largest first, and the eight largest of two sorted eights.
__device__ __forceinline__ void swap_desc(int& a, int& b) {
    const int hi = max(a, b);
    b = min(a, b);
    a = hi;
}
__device__ __forceinline__ void sort8(int (&k)[8]) {
#define MOE_CE(i, j) swap_desc(k[i], k[j])
    MOE_CE(0, 1); MOE_CE(2, 3); MOE_CE(4, 5); MOE_CE(6, 7);
    MOE_CE(0, 2); MOE_CE(1, 3); MOE_CE(4, 6); MOE_CE(5, 7);
    MOE_CE(1, 2); MOE_CE(5, 6);
    MOE_CE(0, 4); MOE_CE(1, 5); MOE_CE(2, 6); MOE_CE(3, 7);
    MOE_CE(2, 4); MOE_CE(3, 5);
    MOE_CE(1, 2); MOE_CE(3, 4); MOE_CE(5, 6);
}
__device__ __forceinline__ void merge8(int (&k)[8], const int (&o)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = max(k[i], o[7 - i]);  // the eight largest, bitonic
    MOE_CE(0, 4); MOE_CE(1, 5); MOE_CE(2, 6); MOE_CE(3, 7);
    MOE_CE(0, 2); MOE_CE(1, 3); MOE_CE(4, 6); MOE_CE(5, 7);
    MOE_CE(0, 1); MOE_CE(2, 3); MOE_CE(4, 5); MOE_CE(6, 7);
#undef MOE_CE
}

// The eight largest of eight lanes' sorted eights, one per lane: lane `sub` returns the
// kSlotOfLane[sub]-th largest, and `left` the largest of the rest (each lane's part of it: the
// caller takes the maximum over the lanes). Bitonic merges of pairs, fours and eights of lanes: the
// larger of a_i and b_(7-i) over i are the eight largest of two sorted eights, and each lane of
// a merge takes its share of them, 4, 2 and 1, so that a step moves only those.
//   After the pairs' step lanes 0, 1 hold a pair's eight in order, four each; after the fours'
//   step lanes 0, 3, 1, 2 a four's, two each; after the last lanes 0, 6, 3, 5, 1, 7, 2, 4.
constexpr uint32_t kSlotOfLane = 0x51372640u, kLaneOfSlot = 0x42715360u;  // four bits each
__device__ __forceinline__ int merge_lanes8(const int (&k)[8], int sub, int& left) {
    const bool odd = sub & 1, two = sub & 2;
    int r[4];
    left = INT_MIN;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int o = __shfl_xor_sync(kFull, k[7 - j], 1);
        r[j] = max(k[j], o);
        left = max(left, min(k[j], o));
    }
    int n[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // the odd lane holds positions 7 .. 4
        const int x = odd ? r[3 - j] : r[j], o = __shfl_xor_sync(kFull, x, 1);
        n[j] = odd ? min(x, o) : max(x, o);
    }
    swap_desc(n[0], n[2]);
    swap_desc(n[1], n[3]);
    swap_desc(n[0], n[1]);
    swap_desc(n[2], n[3]);
    int p, q;
    {
        const int o3 = __shfl_xor_sync(kFull, n[3], 3), o2 = __shfl_xor_sync(kFull, n[2], 3);
        p = max(n[0], o3);
        q = max(n[1], o2);
        left = max(left, max(min(n[0], o3), min(n[1], o2)));
        const bool low = odd != two;  // lanes 1 and 2 hold positions 4 .. 7
        const int po = __shfl_xor_sync(kFull, p, 1), qo = __shfl_xor_sync(kFull, q, 1);
        p = low ? min(p, po) : max(p, po);
        q = low ? min(q, qo) : max(q, qo);
        const int px = __shfl_xor_sync(kFull, q, 3), qx = __shfl_xor_sync(kFull, p, 3);
        p = two ? min(p, px) : max(p, px);
        q = two ? min(q, qx) : max(q, qx);
        swap_desc(p, q);
    }
    const int o = __shfl_xor_sync(kFull, q, 6);
    int m = max(p, o);
    left = max(left, min(p, o));
    // positions: lane 0 0, 6 1, 3 2, 5 3, 1 4, 7 5, 2 6, 4 7
    const int slot = (int)(kSlotOfLane >> (4 * sub)) & 7;
    const int o4 = __shfl_xor_sync(kFull, m, 1);
    m = slot & 4 ? min(m, o4) : max(m, o4);
    const int o2 = __shfl_xor_sync(kFull, m, 3);
    m = slot & 2 ? min(m, o2) : max(m, o2);
    const int o1 = __shfl_xor_sync(kFull, m, 6);
    return slot & 1 ? min(m, o1) : max(m, o1);
}

template <int BYTES>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// VEC: rows are 16-byte aligned, and a lane's experts whole 16-byte vectors.
template <int L, int NB, bool LOGIT, bool VEC>
__global__ void __launch_bounds__(kSelWarps * 32, 2) select_kernel(const SelectParams P, const SelectLayout Y) {
    constexpr int NT = 32 / L;
    extern __shared__ __align__(16) float smem[];  // biases, then two buffers of rows per warp
    __shared__ __align__(16) int lists[kSelWarps][kMaxExperts + 32];  // the lanes' keys, eight each; a token's slots
    __shared__ int taken;  // steps of the CTA's run that its warps have taken
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = lane % L;
    const int E = P.E, G = P.n_group, per = E / G, k = P.k;
    const bool sigmoid = P.mode == MOE_MODE_SIGMOID;
    const bool top2 = P.rule == MOE_GROUP_TOP2 && per > 1, sums = top2 && G > 1;
    const int g = sub / Y.lpg, r = sub % Y.lpg;
    const int count = g < G ? max(0, min(Y.vr, per - r * Y.vr)) : 0;
    const int first = count > 0 ? g * per + r * Y.vr : 0;  // idle lanes read the row's start
    const int pitch = (E + 3) / 4 * 4;
    float* const bias = smem;  // (b - base) times the values' scale
    float* const rows = smem + (LOGIT ? 0 : pitch) + warp * 2 * NT * pitch;
    int* const keys = lists[warp];
    int* const slots = lists[warp] + kMaxExperts;

    // The CTA's tokens are a run of steps of NT tokens, which its warps take one by one: a token near
    // a tie delays its warp alone.
    const int64_t steps = (P.T + NT - 1) / NT;
    const int64_t s0 = blockIdx.x * steps / gridDim.x;
    const int n = (int)((blockIdx.x + 1) * steps / gridDim.x - s0);
    auto fetch = [&](int i, int buf) {
        if (i < n) {
            const int64_t t = (s0 + i) * NT;
            const int m = (int)min((int64_t)NT, P.T - t) * E;  // the step's rows are one piece
            const float* src = P.logits + t * E;
            float* dst = rows + buf * NT * pitch;
            if (VEC)
                for (int c = 4 * lane; c < m; c += 128) cp_async<16>(dst + c, src + c);
            else
                for (int c = lane; c < m; c += 32) cp_async<4>(dst + c, src + c);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto take = [&]() {
        int i = 0;
        if (lane == 0) i = atomicAdd(&taken, 1);
        return __shfl_sync(kFull, i, 0);
    };
    int step = warp;  // the first ones without asking
    fetch(step, 0);
    if (threadIdx.x == 0) taken = kSelWarps;
    float base = 0.f, scale = 1.f, range = 1.f;
    bool infinite = false;
    if constexpr (!LOGIT) {
        float b[kMaxExperts / 32];
#pragma unroll
        for (int j = 0; j < kMaxExperts / 32; ++j) b[j] = lane + 32 * j < E ? P.b[lane + 32 * j] : NAN;
        base = bias_base(b, range);
        infinite = range == INFINITY;
        scale = kBelowOne * fast_rcp(range);
#pragma unroll
        for (int j = 0; j < kMaxExperts / 32; ++j)  // one warp's share each
            if (j == warp && lane + 32 * j < E) bias[lane + 32 * j] = (b[j] - base) * scale;
    }
    __syncthreads();
    // lanes of equal banks start at different vectors of their own (the order is free)
    const int nvec = Y.vr / 4;
    const int turn = VEC ? (sub * Y.vr / 32) % nvec : 0;
    const uint32_t mask = L == 32 ? kFull : ((1u << (L % 32)) - 1u) << (lane / L * L);
    const int my_slot = L == 8 ? (int)(kSlotOfLane >> (4 * sub)) & 7 : sub;
    auto slot_lane = [](int slot) { return L == 8 ? (int)(kLaneOfSlot >> (4 * (slot & 7))) & 7 : slot; };
    const int next_lane = slot_lane(my_slot + 1);

    for (int buf = 0; step < n; buf ^= 1) {
        const int ahead = take();
        fetch(ahead, buf ^ 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        const int64_t t0 = (s0 + step) * NT, t = t0 + lane / L;
        const bool live = t < P.T;
        const float* const held = rows + buf * NT * pitch + lane / L * E;  // the token's row
        // four of the lane's logits, from place `at` on (a multiple of 4), as far as there are
        auto load4 = [&](int c, int& at, float (&v)[4]) {
            at = 4 * c;
            if (VEC) {
                int o = c + turn;
                if (o >= nvec) o -= nvec;
                at = 4 * o;
                const float4 u = *reinterpret_cast<const float4*>(held + first + at);
                v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = at + j < count ? held[first + at + j] : -INFINITY;
            }
        };
        const int nload = (Y.vr + 3) / 4;
        bool odd = false;  // not a row for this kernel's arithmetic
        float mx = 0.f, sum = 1.f, inv = 1.f;
        if (LOGIT || !sigmoid) {
            mx = -INFINITY;
            for (int c = 0; c < nload; ++c) {
                int at;
                float v[4];
                load4(c, at, v);
                mx = fmaxf(fmaxf(mx, fmaxf(v[0], v[1])), fmaxf(v[2], v[3]));
            }
            mx = seg_max<L>(mx);
            if (LOGIT) odd = !(fabsf(mx) < 1e5f);  // the keys' offset would round by more than their margin
        }
        if (!sigmoid) {
            sum = 0.f;
            for (int c = 0; c < nload; ++c) {
                int at;
                float v[4];
                load4(c, at, v);
                sum += (fast_exp2(kLog2e * (v[0] - mx)) + fast_exp2(kLog2e * (v[1] - mx))) +
                       (fast_exp2(kLog2e * (v[2] - mx)) + fast_exp2(kLog2e * (v[3] - mx)));
            }
            sum = seg_sum<L>(count > 0 ? sum : 0.f);
            odd |= !(sum < 1e30f) || mx == -INFINITY;  // NaN or infinite logits
            inv = fast_rcp(sum);
        }
        const float es = score_err(sigmoid, inv);
        // a value in the keys: kv x + kc (LOGIT: of the logit; else of the score, plus its bias)
        const float kv = LOGIT ? kBelowOne / kLogitRange : sigmoid ? scale : scale * inv;
        const float kc = LOGIT ? (kLogitRange - mx) * kv : 0.f;
        // units that settle an order: twice the score's error and the three roundings of b - base,
        // its scaling and the sum (u each), and both values' rounding to half a unit
        const int tol = LOGIT ? 3 : 3 + (int)((2.f * es + 6.2f * kU * range) * scale * kUnits);
        int key[8];
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
            if (blk > 0 && 8 * blk >= Y.vr) break;
            int kb[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                int at;
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) kb[4 * h + j] = INT_MIN;
                if (8 * blk + 4 * h >= Y.vr) continue;
                load4(2 * blk + h, at, v);
                const int id = INT_MIN + 1 + first + at;
                float bv[4] = {kc, kc, kc, kc};
                if (!LOGIT) {
                    if (VEC) {
                        const float4 u = *reinterpret_cast<const float4*>(bias + first + at);
                        bv[0] = u.x, bv[1] = u.y, bv[2] = u.z, bv[3] = u.w;
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (at + j < count) bv[j] = bias[first + at + j];
                    }
                    if (sigmoid) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[j] = fast_rcp(1.0f + fast_exp2(-kLog2e * v[j]));
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[j] = fast_exp2(kLog2e * (v[j] - mx));
                    }
                } else if (sums) {  // a NaN's score is -inf in the sum
                    odd |= v[0] != v[0] || v[1] != v[1] || v[2] != v[2] || v[3] != v[3];
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (VEC || at + j < count) kb[4 * h + j] = fixed_key(v[j], kv, bv[j], id + j);
            }
            sort8(kb);
            if (blk == 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) key[j] = kb[j];
            } else {
                merge8(key, kb);
            }
        }
        if (count == 0) {  // idle lanes
#pragma unroll
            for (int j = 0; j < 8; ++j) key[j] = INT_MIN;
        }
        auto publish = [&]() {
            int4* to = reinterpret_cast<int4*>(keys + 8 * lane);
            to[0] = make_int4(key[0], key[1], key[2], key[3]);
            to[1] = make_int4(key[4], key[5], key[6], key[7]);
        };
        bool open = true;  // the lane's group stays
        auto lanes_of = [&](int i) { return L == 32 ? kFull : ((1u << (L % 32)) - 1u) << (i * L); };
        bool groups = false;  // unsettled
        if (G > 1) {
            // a group's score in units; sums of scores without a bias as floats
            int a = key[0], b = key[1];
            float fa = -INFINITY, fb = -INFINITY;
            bool rough = false;
            if (LOGIT && top2) {  // from the logits themselves
                if (count > 0) fa = held[expert_of(a)];
                if (count > 1) fb = held[expert_of(b)];
                if (fb > fa) {
                    const float x = fa;
                    fa = fb;
                    fb = x;
                }
                // the third may be the second's equal but for rounding; clamped ones are unordered
                rough = count > 2 && units_of(b) - units_of(key[2]) <= 3;
            }
            for (int o = 1; o < Y.lpg; o <<= 1) {
                const int oa = __shfl_xor_sync(kFull, a, o), ob = __shfl_xor_sync(kFull, b, o);
                b = max(max(b, ob), min(a, oa));
                a = max(a, oa);
                if (LOGIT && top2) {
                    const float xa = __shfl_xor_sync(kFull, fa, o), xb = __shfl_xor_sync(kFull, fb, o);
                    fb = fmaxf(fmaxf(fb, xb), fminf(fa, xa));
                    fa = fmaxf(fa, xa);
                }
            }
            int gs = top2 ? units_of(a) + units_of(b) : units_of(a);
            if (LOGIT && top2)
                gs = __float_as_int(fast_score(sigmoid, fa, mx, inv) + fast_score(sigmoid, fb, mx, inv));
            int rank = 0;
            for (int h = 0; h < G; ++h) {
                const int x = __shfl_sync(kFull, gs, h * Y.lpg, L);
                rank += x > gs || (x == gs && h < g);
            }
            bool kept = g < G && rank < P.topk_group;
            if (P.topk_group < G) {
                if (top2 && g < G) groups |= units_of(b) == 0;  // a sum that counts a value clamped at 0
                const int lo = seg_min<L>(kept ? gs : INT_MAX);
                const int hi = seg_max<L>(!kept && g < G ? gs : INT_MIN);
                if (LOGIT && top2) {
                    // softmax terms are within 160 u of themselves down to e^-87; logits that the
                    // keys do not tell apart are within 6e-6
                    const float x = __int_as_float(lo), y = __int_as_float(hi);
                    const bool vague = (__ballot_sync(kFull, rough && g < G) & mask) != 0;
                    const float gap = sigmoid ? 2.f * (2.f * kSigmoidErr + kU * x) + (vague ? 26.f * kU : 0.f)
                                              : (322.f + (vague ? 101.f : 0.f)) * kU * x;
                    groups |= !(x - y > gap && x > 1e-30f);
                } else {
                    groups |= lo - hi <= (top2 ? 2 * tol : tol);
                }
            }
            const uint32_t unsettled = LOGIT ? 0u : __ballot_sync(kFull, live && groups && !infinite);
            if (unsettled) {
                publish();
                __syncwarp();
                for (int i = 0; i < NT; ++i) {  // the warp together, one token at a time
                    if (!(unsettled & lanes_of(i))) continue;
                    uint32_t o = 0;
                    const bool ok = settle_groups(P, lane, rows + buf * NT * pitch + i * E, keys + 8 * i * L, Y.lpg,
                                                  __shfl_sync(kFull, tol, i * L), __shfl_sync(kFull, mx, i * L), o);
                    if (ok && lane / L == i) {
                        kept = g < G && ((o >> g) & 1u);
                        groups = false;
                    }
                }
                __syncwarp();
            }
            open = kept;
            if (!kept) {
#pragma unroll
                for (int j = 0; j < 8; ++j) key[j] = INT_MIN;
            }
        }
        const int eighth = key[7];  // of a lane that still counts
        // slot my_slot's key, and the largest one that is in no slot
        int mine, last;
        if (L == 8) {
            mine = merge_lanes8(key, sub, last);
            last = seg_max<L>(last);  // the ninth: what follows slot 7
        } else {  // rounds: the lane that holds the largest key moves its list up
            publish();
            mine = INT_MIN;
            for (int i = 0;; ++i) {
                last = seg_max<L>(key[0]);
                if (i == k) break;
                if (sub == i) mine = last;
                if (key[0] == last) {
#pragma unroll
                    for (int j = 0; j < 7; ++j) key[j] = key[j + 1];
                    key[7] = INT_MIN;
                }
            }
        }
        int my_e = max(expert_of(mine), 0);  // (of a key that is none: not used)
        // each slot's key against the next one's (the last slot's against the best one left)
        int next = __shfl_sync(kFull, mine, lane / L * L + (next_lane < L ? next_lane : 0));
        if (my_slot == L - 1 || (L > 8 && my_slot == k - 1)) next = last;
        const int kth = __shfl_sync(kFull, mine, lane / L * L + slot_lane(k - 1));
        const bool close = my_slot < k && units_of(mine) - units_of(next) <= tol;
        // a lane whose eight are all chosen, or may be, can hold a ninth
        const bool ninth = NB > 1 && count > 8 && units_of(eighth) >= units_of(kth) - tol;
        const uint32_t near = __ballot_sync(kFull, live && (close || ninth));
        uint32_t again = __ballot_sync(kFull, live && (odd || groups || infinite));
        if (near & ~again) {
            const uint32_t deep = __ballot_sync(kFull, ninth);
            if (L == 8) publish();
            __syncwarp();
            const uint32_t stay = __ballot_sync(kFull, open && r == 0);
            auto settle = [&](int i, int nkeys, const int* from) {
                const bool ok = settle_slots<LOGIT>(P, lane, rows + buf * NT * pitch + i * E, from, nkeys,
                                                    __shfl_sync(kFull, units_of(kth) - tol, i * L),
                                                    __shfl_sync(kFull, mx, i * L), slots);
                if (!ok) again |= lanes_of(i);
                else if (lane / L == i && my_slot < k) my_e = slots[my_slot];
                __syncwarp();
            };
            for (int i = 0; i < NT; ++i) {
                if (!(near & lanes_of(i)) || (again & lanes_of(i)) || (deep & lanes_of(i))) continue;
                settle(i, 8 * L, keys + 8 * i * L);
            }
            for (int i = 0; NB > 1 && i < NT; ++i) {  // by all of the token's keys, not eight a lane
                if (!(near & deep & lanes_of(i)) || (again & lanes_of(i))) continue;
                const float kvi = __shfl_sync(kFull, kv, i * L), kci = __shfl_sync(kFull, kc, i * L);
                const float mxi = __shfl_sync(kFull, mx, i * L);
                const int nkeys = (E + 31) / 32 * 32;
#pragma unroll 1
                for (int e = lane; e < nkeys; e += 32) {
                    int x = INT_MIN;
                    if (e < E && (G == 1 || ((stay >> (i * L + e / per * Y.lpg)) & 1u))) {
                        const float v = rows[buf * NT * pitch + i * E + e];
                        x = LOGIT ? fixed_key(v, kvi, kci, INT_MIN + 1 + e)
                                  : fixed_key(fast_score(sigmoid, v, mxi, 1.f), kvi, bias[e], INT_MIN + 1 + e);
                    }
                    keys[e] = x;
                }
                __syncwarp();
                settle(i, nkeys, keys);
            }
        }
        finish<L>(P, t, my_slot, live && !(again & mask), my_e, held[my_e], mx, sum);
        if (again) {
            const uint32_t strange = __ballot_sync(kFull, live && (odd || infinite));
            for (int i = 0; i < NT; ++i) {
                const uint32_t m = lanes_of(i);
                if (!(again & m) || t0 + i >= P.T) continue;
                if (LOGIT && !(strange & m)) select_logits(P, t0 + i, lane, rows + buf * NT * pitch + i * E);
                else select_token(P, t0 + i, lane);
            }
        }
        step = ahead;
        __syncwarp();  // the buffer's readers are done before the next copies into it
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
// whole, since the tokens' rows are one piece of memory. 65,536 x 256 sigmoid (73 MB): 13.5 us, 0.80
// of a copy of its bytes; softmax without renormalised gates, where the logits are read too, 26.6
// us, 0.78; 32,768 x 128 of that (37 MB) 9.0 us, 0.60, the rest being launch and first loads. Four
// CTAs per SM and no more, 64 registers: at three 27.4 and 10.0 us, at five with spills 37.8 and 14.5.
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

constexpr int kBwdCtas = 4;  // per SM

template <int L, bool DENSE>
__global__ void __launch_bounds__(kSelWarps * 32, kBwdCtas) select_bwd_kernel(const SelectBwdParams P) {
    constexpr int NT = 32 / L;
    extern __shared__ __align__(16) float rows[];
    __shared__ float token_c[kSelWarps][NT], token_lse[kSelWarps][NT];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = lane % L;
    const int E = P.E, k = P.k;
    // one warp's rows; a multiple of 16 bytes
    float* row = rows + (size_t)warp * ((NT * E + 3) / 4 * 4);
    const bool softmax = P.mode == MOE_MODE_SOFTMAX;
    const int64_t stride = (int64_t)gridDim.x * kSelWarps * NT;
    int e = -1;
    float s = 0.f, dg = 0.f, lse = 0.f;
    auto load = [&](int64_t t0) {  // a token's slots, ahead of their use
        const int64_t t = t0 + lane / L;
        e = -1;
        s = dg = 0.f;
        if (t < P.T && sub < k) {
            e = P.idx[t * k + sub];
            s = P.score[t * k + sub];
            dg = P.dg[t * k + sub];
        }
        if (DENSE && t < P.T && sub == 0) lse = P.lse[t];
    };
    int64_t t0 = ((int64_t)blockIdx.x * kSelWarps + warp) * NT;
    load(t0);
    for (; t0 < P.T; t0 += stride) {
        const int n = (int)min((int64_t)NT, P.T - t0) * E;  // elements of the warp's tokens
        for (int i = 4 * lane; i < n; i += 128)
            *reinterpret_cast<float4*>(row + i) = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t0 + lane / L < P.T && sub < k && (e < 0 || e >= E)) {  // the slot is dropped
            record_error(P.status, MOE_ERR_BAD_INDEX, kSiteSelectBwd);
            e = -1;
            s = dg = 0.f;
        }
        // v = s ds: with renormalised gates from s / S, since 1 / S may leave fp32's range
        float v = P.scale * dg * s;
        if (P.renorm) {
            const float S = seg_sum<L>(s), share = S == 0.f ? 0.f : s / S;
            const float m = seg_sum<L>(share * dg);
            v = P.scale * (dg - m) * share;
        }
        if (DENSE) {
            const float c = P.renorm ? 0.f : seg_sum<L>(v);
            if (sub == 0) {
                token_c[warp][lane / L] = c;
                token_lse[warp][lane / L] = lse;
            }
            if (!P.renorm) v = P.scale * dg;  // p takes the place of s
        }
        if (!softmax) v *= 1.f - s;
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
        load(t0 + stride);
        __syncwarp();
        float* out = P.dlogits + t0 * E;
        const float* extra = P.extra ? P.extra + t0 * E : nullptr;
        const float* l = DENSE ? P.logits + t0 * E : nullptr;
        auto token_of = [&](int i) {
            int q = 0;
#pragma unroll
            for (int h = 1; h < NT; ++h) q += i >= h * E;
            return q;
        };
        // the gradient of a logit x in a token with (lse, sum of s ds) = (lq, cq); `up` = s ds with
        // renormalised gates, else ds
        auto grad = [&](float x, float up, float lq, float cq) {
            if (!DENSE) return up;
            if (lq == -INFINITY) return 0.f;  // no expert has a score
            const float p = fast_exp2(kLog2e * (x - lq));
            return (P.renorm ? up : p * (up - cq)) + P.z_scale * lq * p;
        };
        auto grad_at = [&](int i, float x) {
            const int q = DENSE ? token_of(i) : 0;
            return grad(x, row[i], DENSE ? token_lse[warp][q] : 0.f, DENSE ? token_c[warp][q] : 0.f);
        };
        const bool vec = ((reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(extra) |
                           reinterpret_cast<uintptr_t>(l)) & 15u) == 0;
        const int nv = vec ? n / 4 * 4 : 0;
        for (int i0 = 4 * lane; i0 < nv; i0 += 512) {  // four vectors' loads in flight
            float4 x[4], y[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                x[u] = y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i0 + 128 * u >= nv) continue;
                if (DENSE) x[u] = *reinterpret_cast<const float4*>(l + i0 + 128 * u);
                if (extra) y[u] = *reinterpret_cast<const float4*>(extra + i0 + 128 * u);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + 128 * u;
                if (i >= nv) continue;
                float4 g;
                if (DENSE && E % 4 != 0) {  // a vector may lie in two tokens
                    g = make_float4(grad_at(i, x[u].x), grad_at(i + 1, x[u].y), grad_at(i + 2, x[u].z),
                                    grad_at(i + 3, x[u].w));
                } else {
                    const int q = DENSE ? token_of(i) : 0;
                    const float lq = DENSE ? token_lse[warp][q] : 0.f, cq = DENSE ? token_c[warp][q] : 0.f;
                    const float4 up = *reinterpret_cast<const float4*>(row + i);
                    g = make_float4(grad(x[u].x, up.x, lq, cq), grad(x[u].y, up.y, lq, cq),
                                    grad(x[u].z, up.z, lq, cq), grad(x[u].w, up.w, lq, cq));
                }
                g.x += y[u].x, g.y += y[u].y, g.z += y[u].z, g.w += y[u].w;
                *reinterpret_cast<float4*>(out + i) = g;
            }
        }
        for (int i = nv + lane; i < n; i += 32) {
            const float g = grad_at(i, DENSE ? l[i] : 0.f);
            out[i] = extra ? g + extra[i] : g;
        }
        __syncwarp();  // the rows' readers are done
    }
}

template <int L, int NB>
int launch_lanes(const SelectParams& P, const SelectLayout& Y, bool vec, cudaStream_t st) {
    constexpr int NT = 32 / L, NBMAX = L == 8 ? 4 : 2;  // (rows of any alignment share one kernel)
    const size_t smem = sizeof(float) * ((P.E + 3) / 4 * 4) * ((P.b ? 1 : 0) + kSelWarps * 2 * NT);
    int64_t blocks = cdiv(P.T, (int64_t)NT);      // one step each, until the GPU is full
    const int64_t cap = (int64_t)sm_count() * 2;  // resident CTAs
    if (blocks > cap) blocks = cap;
    auto kern = vec ? (P.b ? select_kernel<L, NB, false, true> : select_kernel<L, NB, true, true>)
                    : (P.b ? select_kernel<L, NBMAX, false, false> : select_kernel<L, NBMAX, true, false>);
    if (smem > 36 * 1024 &&  // (beside the kernel's own 8 KB)
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return MOE_ERR_LAUNCH;
    kern<<<(unsigned)blocks, kSelWarps * 32, smem, st>>>(P, Y);
    return launch_status();
}

// The lanes of a token: the fewest (8, 16 or 32) that hold its slots and its groups, each group in
// the largest power of two of lanes that fits, at up to 32, 16 or 16 experts a lane. 32 lanes hold
// every grouping: n_group lpg > 16 then, so a lane has at most 256 / 17 < 16 experts.
int launch_select(const SelectParams& P, cudaStream_t st) {
    const int per = P.E / P.n_group;
    SelectLayout Y{};
    // few tokens: a warp each, up to one for every resident warp (one token of 256 experts: 3.9 us,
    // 4.6 with eight lanes)
    int L = P.T <= (int64_t)sm_count() * 2 * kSelWarps ? 32 : 8;
    for (;; L *= 2) {
        if (L < 32 && (L < P.k || L < P.n_group)) continue;
        for (Y.lpg = 1; P.n_group * Y.lpg * 2 <= L;) Y.lpg *= 2;
        Y.vr = (int)cdiv(per, Y.lpg);
        // the open lanes list twice the slots: one that lists all of a token's experts may hide
        // others (65,536 x 256, top-8 of one group of 32: 53 us with 16 lanes, 171 with 8)
        const bool listed = Y.vr <= 8 || 8 * P.topk_group * Y.lpg >= 2 * P.k;
        if (L == 32 || (Y.vr <= (L == 8 ? 32 : 16) && listed)) break;
    }
    const bool vec = P.E % 4 == 0 && Y.vr % 4 == 0 && per % Y.vr == 0 && aligned16(P.logits);
    const int nb = Y.vr <= 8 ? 1 : Y.vr <= 16 ? 2 : 4;
    if (L == 8)
        return nb == 1   ? launch_lanes<8, 1>(P, Y, vec, st)
               : nb == 2 ? launch_lanes<8, 2>(P, Y, vec, st)
                         : launch_lanes<8, 4>(P, Y, vec, st);
    if (L == 16) return nb == 1 ? launch_lanes<16, 1>(P, Y, vec, st) : launch_lanes<16, 2>(P, Y, vec, st);
    return nb == 1 ? launch_lanes<32, 1>(P, Y, vec, st) : launch_lanes<32, 2>(P, Y, vec, st);
}

template <int L>
int launch_bwd_lanes(const SelectBwdParams& P, bool dense, cudaStream_t st) {
    constexpr int NT = 32 / L;
    const size_t smem = sizeof(float) * kSelWarps * ((NT * P.E + 3) / 4 * 4);  // 32 KB at most
    int64_t blocks = cdiv(P.T, (int64_t)kSelWarps * NT);
    const int64_t cap = (int64_t)sm_count() * kBwdCtas;
    if (blocks > cap) blocks = cap;
    auto kern = dense ? select_bwd_kernel<L, true> : select_bwd_kernel<L, false>;
    kern<<<(unsigned)blocks, kSelWarps * 32, smem, st>>>(P);
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
    return k <= 8    ? launch_bwd_lanes<8>(P, dense, st)
           : k <= 16 ? launch_bwd_lanes<16>(P, dense, st)
                     : launch_bwd_lanes<32>(P, dense, st);
}
