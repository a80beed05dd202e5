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

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// Softmax statistics of a row: its largest logit (NaN set aside) and the sum of e^(l - max). A
// row whose logits are all -inf has sum 0.
__device__ __forceinline__ void row_softmax(const float* row, int E, int lane, float& mx, float& sum) {
    mx = -INFINITY;
    for (int e = lane; e < E; e += 32) mx = fmaxf(mx, row[e]);
    mx = warp_max(mx);
    sum = 0.f;
    bool bad = false;
    for (int e = lane; e < E; e += 32) {
        const float l = row[e];
        bad |= l != l;
        if (mx != -INFINITY) sum += expf(l - mx);
    }
    sum = warp_sum(sum);
    if (__any_sync(kFull, bad)) sum = NAN;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// Below this sum of the chosen scores one of them may have left fp32's normal range without its
// gate doing so: the gates are then formed in 64 bits.
constexpr float kSmallSum = 9.5367432e-7f;  // 2^-20

// Scores and gates of the chosen experts (lane i < k holds slot i's expert), stored with the
// indices. A token whose chosen scores are all zero (in 64 bits) has gates of zero.
__device__ __forceinline__ void finish(const SelectParams& P, int64_t t, int lane, int my_e,
                                       float mx, float sum) {
    const bool on = lane < P.k, sigmoid = P.mode == MOE_MODE_SIGMOID;
    float l = 0.f, s = 0.f;
    if (on) {
        l = P.logits[t * P.E + my_e];
        s = sigmoid ? stable_sigmoid(l) : sum == 0.f ? 0.f : expf(l - mx) / sum;
    }
    float g = s;
    if (P.renorm) {
        const float S = warp_sum(s);
        if (S < kSmallSum) {
            double sd = 0.0;
            if (on) sd = sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : sum == 0.f ? 0.0 : exp((double)l - (double)mx);
            const double Sd = warp_sum(sd);
            g = Sd == 0.0 ? 0.f : (float)(sd / Sd);
        } else {
            g = s / S;
        }
    }
    if (on) {
        P.idx[t * P.k + lane] = my_e;
        P.gate[t * P.k + lane] = P.scale * g;
        P.score[t * P.k + lane] = s;
    }
    if (P.mode == MOE_MODE_SOFTMAX && P.lse && lane == 0) P.lse[t] = mx + logf(sum);
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
    if (P.mode == MOE_MODE_SOFTMAX) {
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
        s[j] = P.mode == MOE_MODE_SOFTMAX ? s[j] / total : 1.0 / (1.0 + exp(-l));
        if (P.b) s[j] += (double)P.b[e];
        s[j] = no_nan(s[j]);
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

// One warp per token.
__global__ void __launch_bounds__(kSelWarps * 32) select_exact_kernel(const SelectParams P) {
    const int lane = threadIdx.x % 32;
    const int64_t t = (int64_t)blockIdx.x * kSelWarps + threadIdx.x / 32;
    if (t >= P.T) return;  // whole warp
    float mx = 0.f, sum = 1.f;
    if (P.mode == MOE_MODE_SOFTMAX) row_softmax(P.logits + t * P.E, P.E, lane, mx, sum);
    const int my_e = select_exact(P, t, lane, mx);
    finish(P, t, lane, my_e, mx, sum);
}

// ---------------------------------------------------------------------------- backward
// ds_i = scale / S (dg_i - sum_j (s_j / S) dg_j) with renormalised gates (0 where S is 0), else
// scale dg_i. Sigmoid: dl = ds_i s_i (1 - s_i) on the chosen experts. Softmax: dl_e = p_e
// (ds_e - sum_i s_i ds_i), ds_e zero off the chosen experts; with renormalised gates that sum
// is zero, so only the chosen experts have a gradient. z-loss: + (2 z_coef / T) lse p_e.
// One warp per token, lane i < k holding slot i.
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

__global__ void __launch_bounds__(kSelWarps * 32) select_bwd_kernel(const SelectBwdParams P) {
    const int lane = threadIdx.x % 32;
    const int64_t t = (int64_t)blockIdx.x * kSelWarps + threadIdx.x / 32;
    if (t >= P.T) return;  // whole warp
    const int E = P.E, k = P.k;
    const bool softmax = P.mode == MOE_MODE_SOFTMAX;
    int my_e = -1;
    float s = 0.f, dg = 0.f;
    if (lane < k) {
        my_e = P.idx[t * k + lane];
        if (my_e < 0 || my_e >= E) {  // the slot is dropped
            record_error(P.status, MOE_ERR_BAD_INDEX, kSiteSelectBwd);
            my_e = -1;
        } else {
            s = P.score[t * k + lane];
            dg = P.dg[t * k + lane];
        }
    }
    float ds = P.scale * dg;
    if (P.renorm) {
        const float S = warp_sum(s);
        const float m = warp_sum(s / S * dg);
        ds = S == 0.f ? 0.f : P.scale / S * (dg - m);
    }
    const bool dense = softmax && (!P.renorm || P.z_scale != 0.f);
    float c = 0.f, l_se = 0.f;
    if (softmax && !P.renorm) c = warp_sum(s * ds);
    if (dense) l_se = P.lse[t];
    const float v = dense ? ds : softmax ? ds * s : ds * s * (1.f - s);
    for (int e0 = 0; e0 < E; e0 += 32) {  // warp-uniform trip count
        const int e = e0 + lane;
        float up = 0.f;
        for (int i = 0; i < k; ++i) {  // an expert named twice gets both slots' terms
            const int ei = __shfl_sync(kFull, my_e, i);
            const float vi = __shfl_sync(kFull, v, i);
            if (ei == e) up += vi;
        }
        if (e >= E) continue;
        if (dense) {
            if (l_se == -INFINITY) {  // no expert has a score
                up = 0.f;
            } else {
                const float p = expf(P.logits[t * E + e] - l_se);
                up = p * (up - c) + P.z_scale * l_se * p;
            }
        }
        if (P.extra) up += P.extra[t * E + e];
        P.dlogits[t * E + e] = up;
    }
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
    select_exact_kernel<<<(unsigned)cdiv(T, kSelWarps), kSelWarps * 32, 0, (cudaStream_t)stream>>>(P);
    return launch_status();
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
    select_bwd_kernel<<<(unsigned)cdiv(T, kSelWarps), kSelWarps * 32, 0, (cudaStream_t)stream>>>(P);
    return launch_status();
}
