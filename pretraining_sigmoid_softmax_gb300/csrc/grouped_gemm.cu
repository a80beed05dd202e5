// The layer's grouped GEMMs on bf16 and E4M3 operands: configurations of the kernel template of
// grouped_gemm.cuh, and the entry points of the experts' forward and backward.
#include "grouped_gemm.cuh"

namespace moe {
namespace {

// Experts in descending padded row count (ties: lower index), for the weight-gradient
// tile order: the longest reductions are scheduled first.
__global__ void expert_order_kernel(const int64_t* __restrict__ row_offsets, int E,
                                    int32_t* __restrict__ order) {
    const int e = threadIdx.x;
    if (e >= E) return;
    const int64_t ce = row_offsets[e + 1] - row_offsets[e];
    int rank = 0;
    for (int j = 0; j < E; ++j) {
        const int64_t cj = row_offsets[j + 1] - row_offsets[j];
        if (cj > ce || (cj == ce && j < e)) ++rank;
    }
    order[rank] = e;
}

// Configurations of the layer's GEMMs (P: CTA-pair versions).
using CfgG1 = Cfg<128, false, false, true, kEpiSwigluFwd, false, false>;
using CfgG1P = Cfg<128, false, false, true, kEpiSwigluFwd, false, false, true>;
template <int BN> using CfgStoreK = Cfg<BN, false, false, false, kEpiStore, false, false>;
using CfgStoreKP = Cfg<256, false, false, false, kEpiStore, false, false, true>;
// short reductions: sixteen epilogue warps (and 32-column chunks for one output)
using CfgG1P16 = Cfg<128, false, false, true, kEpiSwigluFwd, false, false, true, false, 16, 16>;
using CfgStoreKP32 = Cfg<256, false, false, false, kEpiStore, false, false, true, false, 32, 16>;
template <int BN> using CfgSwigluBwd = Cfg<BN, false, true, false, kEpiSwigluBwd, false, false>;
using CfgSwigluBwdP = Cfg<256, false, true, false, kEpiSwigluBwd, false, false, true>;
using CfgSwigluBwdP16 = Cfg<256, false, true, false, kEpiSwigluBwd, false, false, true, false, 16, 16>;
template <int BN> using CfgDgrad2 = Cfg<BN, false, true, false, kEpiStore, true, false>;
using CfgDgrad2P = Cfg<256, false, true, false, kEpiStore, true, false, true>;
// Reductions this short (K elements) finish their main loop well before eight epilogue warps
// have stored the tile, so those GEMMs take sixteen: G1 (three outputs) up to K = 1024, G2
// (one output, 32-column chunks) up to K = 512. Measured on one box, the small fine-grained
// layer's forward went from 0.156 to 0.137 ms; at K = 768-1024 sixteen warps for G2 (which
// cost an operand stage) were 3% slower, and B4 at K = 512 gained nothing.
constexpr int kShortK = 1024;
constexpr int kShortKOneOut = 512;
constexpr int kShortKB2 = 1024;
template <int BN> using CfgWgrad = Cfg<BN, true, true, false, kEpiStore, false, true>;
using CfgWgradP = Cfg<256, true, true, false, kEpiStore, false, true, true>;
// E4M3 forward GEMMs (rowwise scales)
using CfgG1P8 = Cfg<128, false, false, true, kEpiSwigluFwd, false, false, true, true>;
using CfgStoreKP8 = Cfg<256, false, false, false, kEpiStore, false, false, true, true>;
using CfgStoreK8 = Cfg<128, false, false, false, kEpiStore, false, false, false, true>;
// E4M3 data gradients (B2 on the upstream gradient's codes and W_d's transposed column codes)
using CfgSwigluBwdP8 = Cfg<256, false, false, false, kEpiSwigluBwd, false, false, true, true>;
using CfgSwigluBwd8 = Cfg<128, false, false, false, kEpiSwigluBwd, false, false, false, true>;

}  // namespace

bool make_tmap_bf16_2d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer,
                       uint32_t box_inner, uint32_t box_outer) {
    return make_map(m, base, inner, outer, box_inner, box_outer);
}

bool make_tmap_f32_2d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer,
                      uint32_t box_inner, uint32_t box_outer) {
    auto enc = get_encoder();
    if (!enc || !base) return false;
    cuuint64_t dims[2] = {inner, outer};
    cuuint64_t strides[1] = {inner * 4};
    cuuint32_t box[2] = {box_inner, box_outer};
    cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, box,
               es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_expert_fwd(const moe_bf16* X, const int64_t* row_offsets, int E, int64_t rows,
                              int d, int f, const moe_bf16* W_g, const moe_bf16* W_u,
                              const moe_bf16* W_d, moe_bf16* A, moe_bf16* U, moe_bf16* H,
                              moe_bf16* Y, const float* row_gate, void* ws, size_t ws_bytes,
                              moe_stream_t stream) {
    (void)ws;
    (void)ws_bytes;
    if (!X || !W_g || !W_u || !W_d || !A || !U || !H || !Y) return MOE_ERR_INVALID_ARG;
    if (E <= 0 || rows <= 0 || (!row_offsets && E != 1)) return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts || !gemm_shape_ok(d, f)) return MOE_ERR_UNSUPPORTED;
    const void* ptrs[8] = {X, W_g, W_u, W_d, A, U, H, Y};
    for (const void* p : ptrs)
        if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    if (!device_status_word()) return MOE_ERR_LAUNCH;
    cudaStream_t st = (cudaStream_t)stream;
    CUtensorMap mx, mwg, mwu, mh, mwd;
    if (!make_map(&mx, X, d, rows, 64, 128) || !make_map(&mwg, W_g, d, (uint64_t)E * f, 64, 128) ||
        !make_map(&mwu, W_u, d, (uint64_t)E * f, 64, 128) || !make_map(&mh, H, f, rows, 64, 128))
        return MOE_ERR_LAUNCH;
    // G1: a, u, h
    Params P = base_params(row_offsets, rows, E);
    P.N = f;
    P.K0 = d;
    P.row_scale = row_gate;
    CUtensorMap moa[3], moy[3];
    if (!out_maps(moa, A, U, H, f, rows) || !out_maps(moy, Y, nullptr, nullptr, d, rows))
        return MOE_ERR_LAUNCH;
    int rc = d <= kShortK
                 ? launch<CfgG1P16>(mx, mx, mwg, mwu, P, token_tiles_max(rows, f, 128), st, moa)
                 : launch<CfgG1P>(mx, mx, mwg, mwu, P, token_tiles_max(rows, f, 128), st, moa);
    if (rc != MOE_OK) return rc;
    // G2: y = h W_d^T
    Params Q = base_params(row_offsets, rows, E);
    Q.N = d;
    Q.K0 = f;
    if (d % 256 == 0) {  // CTA pair: each CTA stages 128 of the tile's 256 W_d rows
        if (!make_map(&mwd, W_d, f, (uint64_t)E * d, 64, 128)) return MOE_ERR_LAUNCH;
        if (f <= kShortKOneOut) {
            CUtensorMap moy32[3];
            if (!out_maps(moy32, Y, nullptr, nullptr, d, rows, 32)) return MOE_ERR_LAUNCH;
            rc = launch<CfgStoreKP32>(mh, mh, mwd, mwd, Q, token_tiles_max(rows, d, 256), st, moy32);
        } else {
            rc = launch<CfgStoreKP>(mh, mh, mwd, mwd, Q, token_tiles_max(rows, d, 256), st, moy);
        }
    } else {
        if (!make_map(&mwd, W_d, f, (uint64_t)E * d, 64, 128)) return MOE_ERR_LAUNCH;
        rc = launch<CfgStoreK<128>>(mh, mh, mwd, mwd, Q, token_tiles_max(rows, d, 128), st, moy);
    }
    return rc;
}

static int weight_grads(const moe_bf16* dY, const moe_bf16* X, const moe_bf16* H,
                        const moe_bf16* dA, const moe_bf16* dU, const int64_t* row_offsets, int E,
                        int64_t rows, int d, int f, int32_t* order, moe_bf16* dW_g, moe_bf16* dW_u,
                        moe_bf16* dW_d, cudaStream_t st);

extern "C" int moe_expert_bwd(const moe_bf16* dY, const moe_bf16* X, const moe_bf16* A,
                              const moe_bf16* U, const moe_bf16* H, const int64_t* row_offsets,
                              int E, int64_t rows, int d, int f, const moe_bf16* W_g,
                              const moe_bf16* W_u, const moe_bf16* W_d, moe_bf16* dX,
                              moe_bf16* dA, moe_bf16* dU, moe_bf16* dW_g, moe_bf16* dW_u,
                              moe_bf16* dW_d, const float* row_gate, float* gate_part, int parts,
                              const float* dl_rows, const float* W_r, void* ws, size_t ws_bytes,
                              moe_stream_t stream) {
    if (!dY || !X || !A || !U || !H || !W_g || !W_u || !W_d || !dX || !dA || !dU || !dW_g ||
        !dW_u || !dW_d)
        return MOE_ERR_INVALID_ARG;
    if ((row_gate == nullptr) != (gate_part == nullptr)) return MOE_ERR_INVALID_ARG;
    if (parts <= 0 || parts > MOE_BWD_ALL) return MOE_ERR_INVALID_ARG;
    if ((dl_rows == nullptr) != (W_r == nullptr)) return MOE_ERR_INVALID_ARG;
    if (W_r && (!row_offsets || !aligned16(W_r))) return MOE_ERR_INVALID_ARG;
    if (E <= 0 || rows <= 0 || (!row_offsets && E != 1)) return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts || !gemm_shape_ok(d, f)) return MOE_ERR_UNSUPPORTED;
    const void* ptrs[14] = {dY, X, A, U, H, W_g, W_u, W_d, dX, dA, dU, dW_g, dW_u, dW_d};
    for (const void* p : ptrs)
        if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    if (!device_status_word()) return MOE_ERR_LAUNCH;
    WsCarver wc(ws, ws_bytes);
    int32_t* order = wc.take<int32_t>(E + 1);
    if (row_offsets && (!ws || !wc.ok())) return MOE_ERR_WORKSPACE;
    cudaStream_t st = (cudaStream_t)stream;
    int rc;

    // B2: dH = dY W_d (W_d[e] is [d, f]: K = d rows, N = f contiguous), SwiGLU backward; the
    // saved a and u are staged by TMA (their maps ride in the second A and B slots)
    if (parts & MOE_BWD_DH) {
        constexpr CUtensorMapSwizzle kAuSwz = kAuCols == 32   ? CU_TENSOR_MAP_SWIZZLE_64B
                                              : kAuCols == 16 ? CU_TENSOR_MAP_SWIZZLE_32B
                                                              : CU_TENSOR_MAP_SWIZZLE_NONE;
        CUtensorMap mdy, mwd, msa, msu;
        if (!make_map(&mdy, dY, d, rows, 64, 128) || !make_map(&mwd, W_d, f, (uint64_t)E * d, 64, 64) ||
            !make_map(&msa, A, f, rows, kAuCols, 32, false, kAuSwz) ||
            !make_map(&msu, U, f, rows, kAuCols, 32, false, kAuSwz))
            return MOE_ERR_LAUNCH;
        Params P = base_params(row_offsets, rows, E);
        P.N = f;
        P.K0 = d;
        P.kb_per_expert = d;
        P.ld_out = f;
        P.row_scale = row_gate;
        P.gate_part = gate_part;
        CUtensorMap mod[3];
        if (!out_maps(mod, dA, dU, nullptr, f, rows)) return MOE_ERR_LAUNCH;
        if (f % 256 == 0 && d <= kShortKB2)
            rc = launch<CfgSwigluBwdP16>(mdy, msa, mwd, msu, P, token_tiles_max(rows, f, 256), st, mod);
        else if (f % 256 == 0)
            rc = launch<CfgSwigluBwdP>(mdy, msa, mwd, msu, P, token_tiles_max(rows, f, 256), st, mod);
        else
            rc = launch<CfgSwigluBwd<128>>(mdy, msa, mwd, msu, P, token_tiles_max(rows, f, 128), st,
                                           mod);
        if (rc != MOE_OK) return rc;
    }
    // B4: dX = dA W_g + dU W_u (W_g[e] is [f, d]: K = f rows, N = d contiguous), plus each
    // row's router term when given
    if (parts & MOE_BWD_DX) {
        CUtensorMap mda, mdu, mwg, mwu;
        if (!make_map(&mda, dA, f, rows, 64, 128) || !make_map(&mdu, dU, f, rows, 64, 128) ||
            !make_map(&mwg, W_g, d, (uint64_t)E * f, 64, 64) ||
            !make_map(&mwu, W_u, d, (uint64_t)E * f, 64, 64))
            return MOE_ERR_LAUNCH;
        Params P = base_params(row_offsets, rows, E);
        P.N = d;
        P.K0 = f;
        P.K1 = f;
        P.kb_per_expert = f;
        P.r1_row = dl_rows;
        P.r1_col = W_r;
        CUtensorMap mox[3];
        if (!out_maps(mox, dX, nullptr, nullptr, d, rows)) return MOE_ERR_LAUNCH;
        if (d % 256 == 0)
            rc = launch<CfgDgrad2P>(mda, mdu, mwg, mwu, P, token_tiles_max(rows, d, 256), st, mox);
        else
            rc = launch<CfgDgrad2<128>>(mda, mdu, mwg, mwu, P, token_tiles_max(rows, d, 128), st, mox);
        if (rc != MOE_OK) return rc;
    }
    if (!(parts & MOE_BWD_W)) return MOE_OK;
    return weight_grads(dY, X, H, dA, dU, row_offsets, E, rows, d, f, order, dW_g, dW_u, dW_d, st);
}

// B3 and B5, the weight gradients, from bf16 operands (shared by both expert backward
// entry points): experts scheduled longest first.
static int weight_grads(const moe_bf16* dY, const moe_bf16* X, const moe_bf16* H,
                        const moe_bf16* dA, const moe_bf16* dU, const int64_t* row_offsets, int E,
                        int64_t rows, int d, int f, int32_t* order, moe_bf16* dW_g, moe_bf16* dW_u,
                        moe_bf16* dW_d, cudaStream_t st) {
    int rc;
    if (row_offsets) {
        expert_order_kernel<<<1, kMaxExperts, 0, st>>>(row_offsets, E, order);
        if (launch_status() != MOE_OK) return MOE_ERR_LAUNCH;
    }
    const int32_t* order_ptr = row_offsets ? order : nullptr;
    // B3: dW_d[e] = dY_e^T H_e  (M = d, N = f, K = the expert's rows)
    {
        CUtensorMap mdy, mh;
        if (!make_map(&mdy, dY, d, rows, 64, 64) || !make_map(&mh, H, f, rows, 64, 64))
            return MOE_ERR_LAUNCH;
        Params P = base_params(row_offsets, rows, E);
        P.expert_order = order_ptr;
        P.N = f;
        P.M_out = d;
        P.nprob = 1;
        P.out0 = reinterpret_cast<__nv_bfloat16*>(dW_d);
        const int64_t pair_tiles = (int64_t)E * (d / 256) * (f / 256);
        if (d % 256 == 0 && f % 256 == 0 && 2 * pair_tiles >= sm_count())
            rc = launch<CfgWgradP>(mdy, mdy, mh, mh, P, pair_tiles, st);
        else if (f % 256 == 0 && !(d % 256 == 0 && 2 * pair_tiles < sm_count()))
            rc = launch<CfgWgrad<256>>(mdy, mdy, mh, mh, P, (int64_t)E * (d / BM) * (f / 256), st);
        else  // also when there are few pair tiles: 128-wide tiles on 4x the SMs
            rc = launch<CfgWgrad<128>>(mdy, mdy, mh, mh, P, (int64_t)E * (d / BM) * (f / 128), st);
        if (rc != MOE_OK) return rc;
    }
    // B5: dW_g[e] = dA_e^T X_e, dW_u[e] = dU_e^T X_e  (M = f, N = d)
    {
        CUtensorMap mda, mdu, mxx;
        if (!make_map(&mda, dA, f, rows, 64, 64) || !make_map(&mdu, dU, f, rows, 64, 64) ||
            !make_map(&mxx, X, d, rows, 64, 64))
            return MOE_ERR_LAUNCH;
        Params P = base_params(row_offsets, rows, E);
        P.expert_order = order_ptr;
        P.N = d;
        P.M_out = f;
        P.nprob = 2;
        P.out0 = reinterpret_cast<__nv_bfloat16*>(dW_g);
        P.out1 = reinterpret_cast<__nv_bfloat16*>(dW_u);
        const int64_t pair_tiles = (int64_t)E * 2 * (f / 256) * (d / 256);
        if (d % 256 == 0 && f % 256 == 0 && 2 * pair_tiles >= sm_count())
            rc = launch<CfgWgradP>(mda, mdu, mxx, mxx, P, pair_tiles, st);
        else if (d % 256 == 0 && f % 256 == 0)  // few pair tiles: 128-wide tiles on 4x the SMs
            rc = launch<CfgWgrad<128>>(mda, mdu, mxx, mxx, P, (int64_t)E * 2 * (f / BM) * (d / 128), st);
        else if (d % 256 == 0)
            rc = launch<CfgWgrad<256>>(mda, mdu, mxx, mxx, P, (int64_t)E * 2 * (f / BM) * (d / 256), st);
        else
            rc = launch<CfgWgrad<128>>(mda, mdu, mxx, mxx, P, (int64_t)E * 2 * (f / BM) * (d / 128), st);
    }
    return rc;
}

extern "C" int moe_expert_bwd_fp8(const uint8_t* dYq, const float* sdY, const moe_bf16* dY,
                                  const moe_bf16* X, const moe_bf16* A, const moe_bf16* U,
                                  const moe_bf16* H, const int64_t* row_offsets, int E,
                                  int64_t rows, int d, int f, const uint8_t* Wdq, const float* sWd,
                                  const uint8_t* Wguq, const float* sWgu, moe_bf16* dX,
                                  moe_bf16* dA, moe_bf16* dU, uint8_t* AUq, float* sAU,
                                  moe_bf16* dW_g, moe_bf16* dW_u, moe_bf16* dW_d,
                                  const float* dl_rows, const float* W_r, void* ws,
                                  size_t ws_bytes, moe_stream_t stream) {
    if (!dYq || !sdY || !dY || !X || !A || !U || !H || !Wdq || !sWd || !Wguq || !sWgu || !dX ||
        !dA || !dU || !AUq || !sAU || !dW_g || !dW_u || !dW_d)
        return MOE_ERR_INVALID_ARG;
    if ((dl_rows == nullptr) != (W_r == nullptr)) return MOE_ERR_INVALID_ARG;
    if (W_r && (!row_offsets || !aligned16(W_r))) return MOE_ERR_INVALID_ARG;
    if (E <= 0 || rows <= 0 || (!row_offsets && E != 1)) return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts || !gemm_shape_ok(d, f)) return MOE_ERR_UNSUPPORTED;
    const void* ptrs[14] = {dYq, dY, X, A, U, H, Wdq, Wguq, dX, dA, dU, AUq, dW_g, dW_u};
    for (const void* p : ptrs)
        if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(dW_d) || !aligned16(sWd) || !aligned16(sWgu)) return MOE_ERR_INVALID_ARG;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    if (!device_status_word()) return MOE_ERR_LAUNCH;
    WsCarver wc(ws, ws_bytes);
    int32_t* order = wc.take<int32_t>(E + 1);
    if (row_offsets && (!ws || !wc.ok())) return MOE_ERR_WORKSPACE;
    cudaStream_t st = (cudaStream_t)stream;
    int rc;
    // B2 on E4M3: r = (dy codes)(W_d column codes, transposed: [E f, d], K-major) times the
    // row and column scales, then the SwiGLU backward on the staged bf16 a and u
    {
        constexpr CUtensorMapSwizzle kAuSwz = kAuCols == 32   ? CU_TENSOR_MAP_SWIZZLE_64B
                                              : kAuCols == 16 ? CU_TENSOR_MAP_SWIZZLE_32B
                                                              : CU_TENSOR_MAP_SWIZZLE_NONE;
        CUtensorMap mdy, mwd, msa, msu;
        if (!make_map(&mdy, dYq, d, rows, 128, 128, true) ||
            !make_map(&mwd, Wdq, d, (uint64_t)E * f, 128, 128, true) ||
            !make_map(&msa, A, f, rows, kAuCols, 32, false, kAuSwz) ||
            !make_map(&msu, U, f, rows, kAuCols, 32, false, kAuSwz))
            return MOE_ERR_LAUNCH;
        Params P = base_params(row_offsets, rows, E);
        P.N = f;
        P.K0 = d;
        P.ld_out = f;
        P.sa = sdY;
        P.sb0 = sWd;
        CUtensorMap mod[3];
        if (!out_maps(mod, dA, dU, nullptr, f, rows)) return MOE_ERR_LAUNCH;
        if (f % 256 == 0)
            rc = launch<CfgSwigluBwdP8>(mdy, msa, mwd, msu, P, token_tiles_max(rows, f, 256), st, mod);
        else
            rc = launch<CfgSwigluBwd8>(mdy, msa, mwd, msu, P, token_tiles_max(rows, f, 128), st, mod);
        if (rc != MOE_OK) return rc;
    }
    // [dA | dU] rows -> E4M3 codes under one scale per row (2 f bytes per row)
    rc = launch_quantize_rows_fp8(reinterpret_cast<const __nv_bfloat16*>(dA),
                                  row_offsets ? row_offsets + E : nullptr, rows, f, AUq, sAU, st,
                                  reinterpret_cast<const __nv_bfloat16*>(dU));
    if (rc != MOE_OK) return rc;
    // B4 on E4M3: dX = [dA | dU] codes ([rows, 2f]) x ([W_g; W_u] column codes, transposed:
    // [E d, 2f], K-major), one product over K = 2f, times the row and column scales
    {
        CUtensorMap mau, mwgu;
        if (!make_map(&mau, AUq, 2 * (uint64_t)f, rows, 128, 128, true) ||
            !make_map(&mwgu, Wguq, 2 * (uint64_t)f, (uint64_t)E * d, 128, 128, true))
            return MOE_ERR_LAUNCH;
        Params P = base_params(row_offsets, rows, E);
        P.N = d;
        P.K0 = 2 * f;
        P.sa = sAU;
        P.sb0 = sWgu;
        P.r1_row = dl_rows;
        P.r1_col = W_r;
        CUtensorMap mox[3];
        if (!out_maps(mox, dX, nullptr, nullptr, d, rows)) return MOE_ERR_LAUNCH;
        if (d % 256 == 0)
            rc = launch<CfgStoreKP8>(mau, mau, mwgu, mwgu, P, token_tiles_max(rows, d, 256), st, mox);
        else
            rc = launch<CfgStoreK8>(mau, mau, mwgu, mwgu, P, token_tiles_max(rows, d, 128), st, mox);
        if (rc != MOE_OK) return rc;
    }
    return weight_grads(dY, X, H, dA, dU, row_offsets, E, rows, d, f, order, dW_g, dW_u, dW_d, st);
}

extern "C" int moe_expert_fwd_fp8(const uint8_t* Xq, const float* sX, const int64_t* row_offsets,
                                  int E, int64_t rows, int d, int f, const uint8_t* Wgq,
                                  const float* sWg, const uint8_t* Wuq, const float* sWu,
                                  const uint8_t* Wdq, const float* sWd, moe_bf16* A, moe_bf16* U,
                                  moe_bf16* H, uint8_t* Hq, float* sH, moe_bf16* Y,
                                  const float* row_gate, void* ws, size_t ws_bytes,
                                  moe_stream_t stream) {
    (void)ws;
    (void)ws_bytes;
    if (!Xq || !sX || !Wgq || !sWg || !Wuq || !sWu || !Wdq || !sWd || !A || !U || !H || !Hq ||
        !sH || !Y)
        return MOE_ERR_INVALID_ARG;
    if (E <= 0 || rows <= 0 || (!row_offsets && E != 1)) return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts || !gemm_shape_ok(d, f)) return MOE_ERR_UNSUPPORTED;
    const void* ptrs[9] = {Xq, Wgq, Wuq, Wdq, A, U, H, Hq, Y};
    for (const void* p : ptrs)
        if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    if (!device_status_word()) return MOE_ERR_LAUNCH;
    cudaStream_t st = (cudaStream_t)stream;
    CUtensorMap mx, mwg, mwu, mh, mwd;
    if (!make_map(&mx, Xq, d, rows, 128, 128, true) ||
        !make_map(&mwg, Wgq, d, (uint64_t)E * f, 128, 128, true) ||
        !make_map(&mwu, Wuq, d, (uint64_t)E * f, 128, 128, true) ||
        !make_map(&mh, Hq, f, rows, 128, 128, true) ||
        !make_map(&mwd, Wdq, f, (uint64_t)E * d, 128, 128, true))
        return MOE_ERR_LAUNCH;
    // G1 on E4M3 codes: a, u, h
    Params P = base_params(row_offsets, rows, E);
    P.N = f;
    P.K0 = d;
    P.sa = sX;
    P.sb0 = sWg;
    P.sb1 = sWu;
    P.row_scale = row_gate;
    CUtensorMap moa[3], moy[3];
    if (!out_maps(moa, A, U, H, f, rows) || !out_maps(moy, Y, nullptr, nullptr, d, rows))
        return MOE_ERR_LAUNCH;
    int rc = launch<CfgG1P8>(mx, mx, mwg, mwu, P, token_tiles_max(rows, f, 128), st, moa);
    if (rc != MOE_OK) return rc;
    // h rows -> E4M3 codes for the down projection
    rc = launch_quantize_rows_fp8(reinterpret_cast<const __nv_bfloat16*>(H),
                                  row_offsets ? row_offsets + E : nullptr, rows, f, Hq, sH, st);
    if (rc != MOE_OK) return rc;
    // G2 on E4M3 codes: y
    Params Q = base_params(row_offsets, rows, E);
    Q.N = d;
    Q.K0 = f;
    Q.sa = sH;
    Q.sb0 = sWd;
    if (d % 256 == 0)
        rc = launch<CfgStoreKP8>(mh, mh, mwd, mwd, Q, token_tiles_max(rows, d, 256), st, moy);
    else
        rc = launch<CfgStoreK8>(mh, mh, mwd, mwd, Q, token_tiles_max(rows, d, 128), st, moy);
    return rc;
}

int moe::launch_weight_grads(const moe_bf16* dY, const moe_bf16* X, const moe_bf16* H,
                             const moe_bf16* dA, const moe_bf16* dU, const int64_t* row_offsets,
                             int E, int64_t rows, int d, int f, moe_bf16* dW_g, moe_bf16* dW_u,
                             moe_bf16* dW_d, void* ws, size_t ws_bytes, cudaStream_t st) {
    WsCarver wc(ws, ws_bytes);
    int32_t* order = wc.take<int32_t>(E + 1);
    if (row_offsets && (!ws || !wc.ok())) return MOE_ERR_WORKSPACE;
    return weight_grads(dY, X, H, dA, dU, row_offsets, E, rows, d, f, order, dW_g, dW_u, dW_d, st);
}
