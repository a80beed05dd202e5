// The grouped GEMMs on microscaled 4-bit operands (formats: fp4.cuh; kernel template:
// grouped_gemm.cuh): the plain grouped product, and the experts' forward and backward.
#include "fp4.cuh"
#include "grouped_gemm.cuh"

namespace moe {
namespace {

// Configurations, on CTA pairs where an expert has many rows. 524,288 token rows (532,000 with the padding) of
// 1536 by 4096 columns (MX): 1265 us, 5.2 PFLOP/s; gate and up of 2048 by 768 for 278,000 rows 405 us, 4.7 TB/s;
// SwiGLU backward of the same, with the codes of [dA | dU], 458 us, 5.1 TB/s. MX stages are smaller, so with one output buffer a warp five of
// them fit instead of four, which the loads' latency (1.5 us a round of the stages) is worth: down
// projections of 1536 1544 -> 1270 us, gate and up of 2048 422 -> 371. NV copies twice the scales and
// is bound by that: two output buffers and four stages (sums of 768: 300 us against 330).
template <bool NV>
struct Fp4Gemm {
    static constexpr int QT = NV ? kNvFp4 : kMxFp4;
    using G1 = Cfg<128, false, false, true, kEpiSwigluFwd, false, false, true, QT, 16, 8, !NV>;
    using Store = Cfg<256, false, false, false, kEpiStore, false, false, true, QT, 16, 8, !NV>;
    // outputs that are no multiple of 256 wide: 192 columns (the last tile clipped)
    using Store192 = Cfg<192, false, false, false, kEpiStore, false, false, true, QT, 16, 12>;
    // few rows an expert: one CTA a tile (few_rows below)
    using G1One = Cfg<128, false, false, true, kEpiSwigluFwd, false, false, false, QT, 16, 8, true>;
    using StoreOne = Cfg<128, false, false, false, kEpiStore, false, false, false, QT, 16, 8, true>;
    using Bwd = Cfg<192, false, false, false, kEpiSwigluBwd, false, false, true, QT, 16, 12>;
};

// Whether most experts have one 128-row tile at most: the capacity of T k rows on E experts is T k + 127
// E, so 192 E stands for about 64 rows an expert. A pair's second half would then load and multiply
// rows of other experts, and half as many CTAs would have a tile: one token through experts of 4096 x
// 1536 takes 42 us on single CTAs and 49 on pairs.
bool few_rows(const int64_t* row_offsets, int E, int64_t rows) {
    return row_offsets ? rows <= 192 * (int64_t)E : rows <= BM;
}

// An operand: codes [rows, K / 2], tiled scales and, in NV, the rows' powers of two.
struct Operand {
    const uint8_t* q;
    const uint8_t* s;
    const float* g;
};

// Rows and tiles are counted in 32 bits on the device: of the token rows, the weights' rows and the
// scale tiles (a tensor map's coordinates), and of the output tiles.
bool sizes_ok(int64_t rows, int E, int K, int N) {
    const int64_t most = INT32_MAX - 511;
    const int64_t wide = rows > (int64_t)E * N ? rows : (int64_t)E * N;
    return wide <= most && cdiv(wide, 128) * (K / 64) <= most &&
           (cdiv(rows, BM) + E) * cdiv(N, 128) <= most;
}

bool operand_ok(const Operand& o, int fmt) {
    return o.q && o.s && (fmt == MOE_FP4_NV) == (o.g != nullptr) && aligned16(o.q) && aligned16(o.s) &&
           aligned16(o.g);
}

bool code_map(CUtensorMap* m, const uint8_t* q, int K, uint64_t rows, int box_rows = 128) {
    return make_map(m, q, (uint64_t)K / 2, rows, 128, (uint32_t)box_rows, true);
}

// Scale tiles as rows of 128 32-bit words, SFK of them a box.
template <bool NV>
bool scale_map(CUtensorMap* m, const uint8_t* s, int K, int64_t rows) {
    auto enc = get_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {kSfTile / 4, (cuuint64_t)(cdiv(rows, 128) * (K / Fp4<NV>::TILE_K))};
    cuuint64_t strides[1] = {kSfTile};
    cuuint32_t box[2] = {kSfTile / 4, (cuuint32_t)Fp4Gemm<NV>::Store::SFK};
    cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_INT32, 2, const_cast<uint8_t*>(s), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Y = X W^T for each expert's rows, bf16 out; r1_row / r1_col as in Params.
template <bool NV>
int product(const Operand& X, const int64_t* row_offsets, int E, int64_t rows, int K, int N,
            const Operand& W, moe_bf16* Y, const float* r1_row, const float* r1_col, cudaStream_t st) {
    using G = Fp4Gemm<NV>;
    CUtensorMap mx, mw, sf[3], mo[3];
    const bool one = few_rows(row_offsets, E, rows), wide = N % 256 == 0;
    if (!code_map(&mx, X.q, K, rows) ||
        !code_map(&mw, W.q, K, (uint64_t)E * N, one || wide ? 128 : 96) ||
        !scale_map<NV>(&sf[0], X.s, K, rows) || !scale_map<NV>(&sf[1], W.s, K, (int64_t)E * N) ||
        !out_maps(mo, Y, nullptr, nullptr, N, rows, G::Store::OCOLS))
        return MOE_ERR_LAUNCH;
    sf[2] = sf[1];
    Params P = base_params(row_offsets, rows, E);
    P.N = N;
    P.K0 = K;
    P.sa = X.g;
    P.sb0 = W.g;
    P.r1_row = r1_row;
    P.r1_col = r1_col;
    if (one)
        return launch<typename G::StoreOne>(mx, mx, mw, mw, P, token_tiles_max(rows, N, 128), st, mo, sf);
    if (wide)
        return launch<typename G::Store>(mx, mx, mw, mw, P, token_tiles_max(rows, N, 256), st, mo, sf);
    return launch<typename G::Store192>(mx, mx, mw, mw, P, token_tiles_max(rows, N, 192), st, mo, sf);
}

// a, u = X W_g^T, X W_u^T; h = silu(a) u.
template <bool NV>
int swiglu(const Operand& X, const int64_t* row_offsets, int E, int64_t rows, int d, int f,
           const Operand& Wg, const Operand& Wu, moe_bf16* A, moe_bf16* U, moe_bf16* H, uint8_t* Hq,
           uint8_t* sH, const float* row_gate, cudaStream_t st) {
    using G = Fp4Gemm<NV>;
    CUtensorMap mx, mg, mu, sf[3], mo[3];
    if (!code_map(&mx, X.q, d, rows) || !code_map(&mg, Wg.q, d, (uint64_t)E * f) ||
        !code_map(&mu, Wu.q, d, (uint64_t)E * f) || !scale_map<NV>(&sf[0], X.s, d, rows) ||
        !scale_map<NV>(&sf[1], Wg.s, d, (int64_t)E * f) || !scale_map<NV>(&sf[2], Wu.s, d, (int64_t)E * f) ||
        !out_maps(mo, A ? A : H, U, A ? H : nullptr, f, rows, G::G1::OCOLS))
        return MOE_ERR_LAUNCH;
    Params P = base_params(row_offsets, rows, E);
    P.N = f;
    P.K0 = d;
    P.sa = X.g;
    P.sb0 = Wg.g;
    P.sb1 = Wu.g;
    P.row_scale = row_gate;
    P.only_h = A == nullptr;
    P.oq = Hq;
    P.os = sH;
    if (few_rows(row_offsets, E, rows))
        return launch<typename G::G1One>(mx, mx, mg, mu, P, token_tiles_max(rows, f, 128), st, mo, sf);
    return launch<typename G::G1>(mx, mx, mg, mu, P, token_tiles_max(rows, f, 128), st, mo, sf);
}

// r = dY W_d; da, du from the saved a and u.
template <bool NV>
int swiglu_bwd(const Operand& dY, const moe_bf16* A, const moe_bf16* U, const int64_t* row_offsets,
               int E, int64_t rows, int d, int f, const Operand& Wd, moe_bf16* dA, moe_bf16* dU,
               uint8_t* AUq, uint8_t* sAU, cudaStream_t st) {
    using G = Fp4Gemm<NV>;
    CUtensorMap my, mw, ma, mu, sf[3], mo[3];
    if (!code_map(&my, dY.q, d, rows) || !code_map(&mw, Wd.q, d, (uint64_t)E * f, 96) ||
        !scale_map<NV>(&sf[0], dY.s, d, rows) || !scale_map<NV>(&sf[1], Wd.s, d, (int64_t)E * f) ||
        !make_map(&ma, A, f, rows, G::Bwd::AUC, 32, false, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !make_map(&mu, U, f, rows, G::Bwd::AUC, 32, false, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !out_maps(mo, dA, dU, nullptr, f, rows, G::Bwd::OCOLS))
        return MOE_ERR_LAUNCH;
    static_assert(G::Bwd::AUC == 32, "64-byte rows of the staged a and u");
    sf[2] = sf[1];
    Params P = base_params(row_offsets, rows, E);
    P.N = f;
    P.K0 = d;
    P.ld_out = f;
    P.sa = dY.g;
    P.sb0 = Wd.g;
    P.oq = AUq;
    P.os = sAU;
    return launch<typename G::Bwd>(my, ma, mw, mu, P, token_tiles_max(rows, f, 192), st, mo, sf);
}

int quantize(const moe_bf16* X, const moe_bf16* X1, const int64_t* row_offsets, int E, int64_t rows,
             int cols, int fmt, uint8_t* Q, uint8_t* S, float* g, cudaStream_t st) {
    return launch_quantize_rows_fp4(reinterpret_cast<const __nv_bfloat16*>(X),
                                    reinterpret_cast<const __nv_bfloat16*>(X1),
                                    row_offsets ? row_offsets + E : nullptr, rows, cols, fmt, Q, S, g, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_grouped_gemm_fp4(const uint8_t* Xq, const uint8_t* sX, const float* gX,
                                    const int64_t* row_offsets, int E, int64_t rows, int K, int N,
                                    const uint8_t* Wq, const uint8_t* sW, const float* gW, int fmt,
                                    moe_bf16* Y, moe_stream_t stream) {
    if (fmt != MOE_FP4_MX && fmt != MOE_FP4_NV) return MOE_ERR_INVALID_ARG;
    const Operand X{Xq, sX, gX}, W{Wq, sW, gW};
    if (!operand_ok(X, fmt) || !operand_ok(W, fmt) || !Y || !aligned16(Y)) return MOE_ERR_INVALID_ARG;
    if (E <= 0 || rows <= 0 || (!row_offsets && E != 1)) return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts || !gemm_shape_ok(K, N) || !sizes_ok(rows, E, K, N)) return MOE_ERR_UNSUPPORTED;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    if (!device_status_word()) return MOE_ERR_LAUNCH;
    cudaStream_t st = (cudaStream_t)stream;
    return fmt == MOE_FP4_NV ? product<true>(X, row_offsets, E, rows, K, N, W, Y, nullptr, nullptr, st)
                             : product<false>(X, row_offsets, E, rows, K, N, W, Y, nullptr, nullptr, st);
}

extern "C" int moe_expert_fwd_fp4(const uint8_t* Xq, const uint8_t* sX, const float* gX,
                                  const int64_t* row_offsets, int E, int64_t rows, int d, int f,
                                  const uint8_t* Wgq, const uint8_t* sWg, const float* gWg,
                                  const uint8_t* Wuq, const uint8_t* sWu, const float* gWu,
                                  const uint8_t* Wdq, const uint8_t* sWd, const float* gWd, int fmt,
                                  moe_bf16* A, moe_bf16* U, moe_bf16* H, uint8_t* Hq, uint8_t* sH,
                                  float* gH, moe_bf16* Y, const float* row_gate, moe_stream_t stream) {
    if (fmt != MOE_FP4_MX && fmt != MOE_FP4_NV) return MOE_ERR_INVALID_ARG;
    const Operand X{Xq, sX, gX}, Wg{Wgq, sWg, gWg}, Wu{Wuq, sWu, gWu}, Wd{Wdq, sWd, gWd}, Hc{Hq, sH, gH};
    for (const Operand* o : {&X, &Wg, &Wu, &Wd, &Hc})
        if (!operand_ok(*o, fmt)) return MOE_ERR_INVALID_ARG;
    if ((A == nullptr) != (U == nullptr) || !H || !Y) return MOE_ERR_INVALID_ARG;
    for (const moe_bf16* p : {A, U, H, Y})
        if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
    if (E <= 0 || rows <= 0 || (!row_offsets && E != 1)) return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts || !gemm_shape_ok(d, f) || f > kFp4MaxCols || !sizes_ok(rows, E, d, f) ||
        !sizes_ok(rows, E, f, d))
        return MOE_ERR_UNSUPPORTED;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    if (!device_status_word()) return MOE_ERR_LAUNCH;
    cudaStream_t st = (cudaStream_t)stream;
    const bool nv = fmt == MOE_FP4_NV;
    // MX: the epilogue has whole blocks of h and forms their codes; NV needs the whole row first
    int rc = nv ? swiglu<true>(X, row_offsets, E, rows, d, f, Wg, Wu, A, U, H, nullptr, nullptr, row_gate, st)
                : swiglu<false>(X, row_offsets, E, rows, d, f, Wg, Wu, A, U, H, Hq, sH, row_gate, st);
    if (rc == MOE_OK && nv) rc = quantize(H, nullptr, row_offsets, E, rows, f, fmt, Hq, sH, gH, st);
    if (rc != MOE_OK) return rc;
    return nv ? product<true>(Hc, row_offsets, E, rows, f, d, Wd, Y, nullptr, nullptr, st)
              : product<false>(Hc, row_offsets, E, rows, f, d, Wd, Y, nullptr, nullptr, st);
}

extern "C" int moe_expert_bwd_fp4(const uint8_t* dYq, const uint8_t* sdY, const float* gdY,
                                  const moe_bf16* dY, const moe_bf16* X, const moe_bf16* A,
                                  const moe_bf16* U, const moe_bf16* H, const int64_t* row_offsets,
                                  int E, int64_t rows, int d, int f, const uint8_t* Wdq,
                                  const uint8_t* sWd, const float* gWd, const uint8_t* Wguq,
                                  const uint8_t* sWgu, const float* gWgu, int fmt, moe_bf16* dX,
                                  moe_bf16* dA, moe_bf16* dU, uint8_t* AUq, uint8_t* sAU, float* gAU,
                                  moe_bf16* dW_g, moe_bf16* dW_u, moe_bf16* dW_d, int parts,
                                  const float* dl_rows, const float* W_r, void* ws, size_t ws_bytes,
                                  moe_stream_t stream) {
    if (fmt != MOE_FP4_MX && fmt != MOE_FP4_NV) return MOE_ERR_INVALID_ARG;
    if (parts <= 0 || parts > MOE_BWD_ALL) return MOE_ERR_INVALID_ARG;
    const Operand dYc{dYq, sdY, gdY}, Wd{Wdq, sWd, gWd}, Wgu{Wguq, sWgu, gWgu}, AU{AUq, sAU, gAU};
    if (!dA || !dU || !aligned16(dA) || !aligned16(dU)) return MOE_ERR_INVALID_ARG;
    if ((parts & MOE_BWD_DH) && (!operand_ok(dYc, fmt) || !operand_ok(Wd, fmt) || !A || !U ||
                                 !aligned16(A) || !aligned16(U)))
        return MOE_ERR_INVALID_ARG;
    if ((parts & MOE_BWD_DX) && (!operand_ok(Wgu, fmt) || !operand_ok(AU, fmt) || !dX || !aligned16(dX)))
        return MOE_ERR_INVALID_ARG;
    if (parts & MOE_BWD_W)
        for (const moe_bf16* p : {dY, X, H, (const moe_bf16*)dW_g, (const moe_bf16*)dW_u,
                                  (const moe_bf16*)dW_d})
            if (!p || !aligned16(p)) return MOE_ERR_INVALID_ARG;
    if ((dl_rows == nullptr) != (W_r == nullptr)) return MOE_ERR_INVALID_ARG;
    if (W_r && (!row_offsets || !aligned16(W_r))) return MOE_ERR_INVALID_ARG;
    if (E <= 0 || rows <= 0 || (!row_offsets && E != 1)) return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts || !gemm_shape_ok(d, f) || 2 * (int64_t)f > kFp4MaxCols ||
        !sizes_ok(rows, E, d, f) || !sizes_ok(rows, E, 2 * f, d))
        return MOE_ERR_UNSUPPORTED;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    if (!device_status_word()) return MOE_ERR_LAUNCH;
    cudaStream_t st = (cudaStream_t)stream;
    const bool nv = fmt == MOE_FP4_NV;
    int rc = MOE_OK;
    // MX: dA's and dU's codes are formed where they are written, if this call goes on to use them
    const bool formed = !nv && (parts & MOE_BWD_DH) && (parts & MOE_BWD_DX);
    if (parts & MOE_BWD_DH) {
        rc = nv ? swiglu_bwd<true>(dYc, A, U, row_offsets, E, rows, d, f, Wd, dA, dU, nullptr, nullptr, st)
                : swiglu_bwd<false>(dYc, A, U, row_offsets, E, rows, d, f, Wd, dA, dU,
                                    formed ? AUq : nullptr, formed ? sAU : nullptr, st);
        if (rc != MOE_OK) return rc;
    }
    if (parts & MOE_BWD_DX) {
        if (!formed) rc = quantize(dA, dU, row_offsets, E, rows, f, fmt, AUq, sAU, gAU, st);
        if (rc != MOE_OK) return rc;
        rc = nv ? product<true>(AU, row_offsets, E, rows, 2 * f, d, Wgu, dX, dl_rows, W_r, st)
                : product<false>(AU, row_offsets, E, rows, 2 * f, d, Wgu, dX, dl_rows, W_r, st);
        if (rc != MOE_OK) return rc;
    }
    if (!(parts & MOE_BWD_W)) return MOE_OK;
    return launch_weight_grads(dY, X, H, dA, dU, row_offsets, E, rows, d, f, dW_g, dW_u, dW_d, ws,
                               ws_bytes, st);
}
