// SwiGLU experts as grouped GEMMs on the sm_100-family tensor cores (tcgen05, TMEM, TMA).
//
// "The whole stack, in the open" (Apex-3), "What's inside", row "Fine-grained MoE": the
// experts run as grouped GEMMs. Handbook summary, section 2.5: a bias-free SwiGLU expert
// has three weight matrices (gate, up, down).
//
// One persistent kernel template serves every GEMM of the layer:
//   G1  [a|u] = X W_g^T, X W_u^T      two accumulators, SwiGLU in the epilogue (A, U, H out)
//   G2  Y = H W_d^T
//   B2  dH = dY W_d, SwiGLU backward in the epilogue (dA, dU out)
//   B4  dX = dA W_g + dU W_u          K split over two operand pairs
//   B3  dW_d[e] = dY_e^T H_e           weight gradients: K runs over expert e's rows
//   B5  dW_g[e] = dA_e^T X_e, dW_u[e] = dU_e^T X_e
// Row tiles are 128 rows of the expert-major layout, whose segments are padded to 128
// rows, so every tile belongs to one expert and is found from row_offsets on the device
// (no host synchronisation). Roles per CTA (384 threads, 512 with twelve epilogue warps or 640 with
// sixteen, one CTA per SM):
//   warp 0  TMA producer (one thread): operand tiles into a ring of shared-memory stages;
//   warp 1  MMA issuer (one thread): tcgen05.mma 128 x N x 16 steps into a TMEM accumulator;
//   warp 2  allocates / frees tensor memory (two accumulators, double-buffered);
//   warps 4-11 epilogue: tcgen05.ld of TMEM lanes 0-127 (one output row per thread; warps w
//            and w + 4 share a lane quadrant and take one half of the columns each), the
//            fused elementwise step, bf16 outputs. Token-major outputs (G1, G2, B2, B4) are
//            packed into swizzled shared-memory boxes and written by TMA stores; B2 reads
//            its saved a and u through TMA-staged boxes; weight gradients store per thread.
//            Two warps per quadrant double the loads and stores in flight; bf16 GEMMs with a
//            reduction of at most 1024 (G1) or 512 (G2) take four per quadrant (warps 4-19), as their main
//            loop is shorter than eight warps' epilogue of the previous tile.
// Pair mode (a cluster of two CTAs on two SMs): the leading CTA issues
// tcgen05.mma.cta_group::2 over a 256-row tile; each CTA stages its own 128 rows of A and
// half of the tile's B columns, so per SM the shared-memory operand traffic and the TMA
// bytes per FLOP drop by a third compared with a 128 x 256 tile on one SM. Both CTAs' TMA
// loads complete on the leader's "full" barriers, the leader's commits arrive on both
// CTAs' barriers (multicast), and both epilogues release the accumulator to the leader.
// E2M1 operands (two codes a byte, 256 K elements per 128-byte row) bring the scales of their
// blocks as 512-byte tiles of 128 rows x 4 blocks: TMA copies them beside the operands, two
// threads of their own (warps 2 and 3) put them into tensor memory with tcgen05.cp, a stage
// ahead, and the tensor cores multiply them in (kind::mxf4 with a power of two per 32,
// kind::mxf4nvf4 with an E4M3 scale per 16). Issued by the MMA thread itself the copies and
// the products take turns: a stage of 256 K elements took 0.55 us (MX, 6 copies) and 0.74
// (NV, 12), and takes 0.38 and 0.41 with the two copying threads (what a longer K adds to a 256 x 256
// tile). The scales leave less than two whole accumulators of 256 columns, so the two share a few
// columns (Cfg::OV).
// Operand tiles use the 128-byte swizzle. K-major tiles are TMA boxes of 64 K-elements x
// rows; MN-major tiles are boxes of 64 MN-elements x 64 k-rows. Every wait on an mbarrier
// is bounded in time; a wait that runs out records MOE_ERR_TIMEOUT, stops every role of
// the CTA and the kernel frees its tensor memory before returning.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "common.cuh"
#include "fp4.cuh"
#include "sizes.h"
#include "tmap.h"

namespace moe {
namespace {

constexpr int kMaxDevices = 64;  // as the status words
constexpr int BM = 128;
constexpr int BK = 64;        // bf16 K elements per stage (128 bytes per row)
constexpr int BK_FP8 = 128;   // E4M3 K elements per stage (also 128 bytes per row)
constexpr int BK_FP4 = 256;   // E2M1 K elements per stage (also 128 bytes per row)
constexpr int kSfTile = 512;  // bytes of a scale tile: 128 rows x 4 blocks
constexpr int kEpiWarps = 8;  // default: two per TMEM lane quadrant, each half the columns
constexpr int kSmemBudget = 200 * 1024;

enum Epi : int { kEpiSwigluFwd = 0, kEpiStore = 1, kEpiSwigluBwd = 2 };
// SwiGLU backward: each epilogue warp stages the saved a and u of its 32 rows by TMA, kAuCols
// columns per chunk, kAuBufs chunks deep; the ring of operand stages gets what is left of
// kSmemBudgetAu.
constexpr int kAuCols = 16;
constexpr int kAuBufs = 2;
constexpr int kSmemBudgetAu = 220 * 1024;
constexpr int kSmemBudgetFp4 = 222 * 1024;
// Token-major epilogues stage their outputs in shared memory, 16 columns x 32 rows per warp
// and output, and write them with TMA stores: two buffers deep, or one for the SwiGLU
// backward, whose operand ring then keeps a fifth stage (what bounds it at K = 4096).
constexpr int kOutCols = 16;

// Operand types (Cfg's QT_; 0 and 1 also as false and true).
enum Operands : int { kBf16 = 0, kE4m3 = 1, kMxFp4 = 2, kNvFp4 = 3 };

template <int BN_, bool A_MN_, bool B_MN_, bool DUAL_, int EPI_, bool TWO_K_, bool WGRAD_,
          bool PAIR_ = false, int QT_ = kBf16, int OC_ = kOutCols, int EW_ = kEpiWarps,
          bool DEEP_ = false>
struct Cfg {
    // epilogue warps: 8 (two per TMEM lane quadrant), or 16 for GEMMs whose reduction is so
    // short that the epilogue, not the tensor cores, sets the pace (at most 96 registers); 12
    // for the 192-column tiles of E2M1
    static constexpr int EW = EW_;
    static constexpr int THREADS = 128 + 32 * EW;
    static_assert(EW == 8 || EW == 16 || EW == 12, "epilogue warps");
    static constexpr bool FP8 = QT_ == kE4m3;  // E4M3 operands with row / column scales
    static constexpr bool NV = QT_ == kNvFp4;  // E2M1, E4M3 scale per 16, power of two per row
    static constexpr bool FP4 = QT_ == kMxFp4 || NV;
    static constexpr bool DEEP = DEEP_;  // E2M1: one output buffer a warp, one operand stage more
    static constexpr int KB = FP4 ? BK_FP4 : FP8 ? BK_FP8 : BK;  // K elements per stage
    static constexpr int BN = BN_;           // output columns per tile (per B matrix if DUAL)
    static constexpr bool A_MN = A_MN_;
    static constexpr bool B_MN = B_MN_;
    static constexpr bool DUAL = DUAL_;      // two B operands -> gate and up accumulators (G1)
    static constexpr int EPI = EPI_;
    static constexpr bool TWO_K = TWO_K_;    // K = [K0 from (a0,b0)] ++ [K1 from (a1,b1)]
    static constexpr bool WGRAD = WGRAD_;    // M = weight rows, K = expert's token rows
    static constexpr bool PAIR = PAIR_;      // CTA pair: 256-row tiles, B split between CTAs
    static constexpr int MMA_N = DUAL ? 2 * BN : BN;         // accumulator columns per row
    static constexpr int BROWS = PAIR ? MMA_N / 2 : MMA_N;   // B rows staged by this CTA
    static constexpr int TILE_M = PAIR ? 2 * BM : BM;        // rows of one (pair) tile
    static constexpr int A_BYTES = BM * 128;     // 128-byte rows in either type
    static constexpr int B_BYTES = BROWS * 128;
    // E2M1: tiles of scales per operand row block and stage (a tile spans 128 K elements with
    // blocks of 32, 64 with blocks of 16). Each CTA of a pair takes its own A rows' scales and
    // those of all the tile's B columns.
    static constexpr int SFK = FP4 ? (NV ? 4 : 2) : 0;
    static constexpr int SFB_TILES = (MMA_N + 127) / 128;
    static constexpr int SFA_BYTES = SFK * kSfTile;
    static constexpr int SF_BYTES = SFA_BYTES * (1 + SFB_TILES);
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SF_BYTES;  // this CTA's bytes per K block
    static constexpr bool AU = EPI == kEpiSwigluBwd;
    // staged a and u, and the outputs made of them: 32 columns a chunk for E2M1, whose main loops are
    // so short that the number of TMA rows sets the pace, else 16
    static constexpr int AUC = FP4 ? 32 : kAuCols;
    static constexpr int AU_BUF_BYTES = 2 * 32 * AUC * 2;  // a and u: 32 rows x AUC
    static_assert(!(FP4 && AU) || BN / (EW / 4) == kAuBufs * AUC, "E2M1: a tile's a and u staged whole");
    static constexpr int AU_BYTES = AU ? EW * kAuBufs * AU_BUF_BYTES : 0;
    static constexpr bool TS = !WGRAD;  // token-major outputs leave by TMA stores
    static constexpr int NOUT = EPI == kEpiSwigluFwd ? 3 : EPI == kEpiSwigluBwd ? 2 : 1;
    // output columns per staged chunk: 16, or 32 (single-output epilogues of short-K GEMMs,
    // where the per-chunk fence and store issue dominate) at the same shared-memory size
    // (E2M1: 64 columns a box, whole 128-byte lines, in one or two buffers a warp; see epilogue_fp4)
    static constexpr int OCOLS =  // (E2M1 with AU: from a's and u's own buffers)
        FP4 ? (AU ? AUC : BN / (EW / 4) < 64 ? BN / (EW / 4) : 64) : OC_;
    static_assert(FP4 || OCOLS == 16 || (OCOLS == 32 && NOUT == 1 && !AU), "output chunk width");
    static constexpr int OUT_BOX_BYTES = 32 * OCOLS * 2;             // one output, one chunk
    static constexpr int OUT_BUF_BYTES = (FP4 && !AU ? 1 : NOUT) * OUT_BOX_BYTES;  // one buffer
    static constexpr int OUT_DEPTH =
        FP4 ? (AU || DEEP || EW != 8 ? 1 : 2)
            : (AU || OCOLS == 32 || EW == 16) ? 1 : 2;  // buffers per warp
    static constexpr int OUT_BYTES = TS && !(FP4 && AU) ? EW * OUT_DEPTH * OUT_BUF_BYTES : 0;
    // NV: each epilogue warp's columns' powers of two, fetched while the tile's main loop runs
    static constexpr int CS_FLOATS = NV ? BN / (EW / 4) * (DUAL ? 2 : 1) : 0;
    static constexpr int CS_BYTES = EW * CS_FLOATS * 4;
    static constexpr int BUDGET =
        (FP4 ? kSmemBudgetFp4 : AU || TS ? kSmemBudgetAu : kSmemBudget) - AU_BYTES - OUT_BYTES - CS_BYTES;
    static constexpr int STAGES = (BUDGET / STAGE_BYTES) > 6 ? 6 : (BUDGET / STAGE_BYTES);
    static constexpr int ACC_COLS = MMA_N;
    // E2M1: the scales of a stage take SFC columns of tensor memory, and two stages' lie at its
    // start. With 256-column accumulators the two buffers then share OV columns: the last
    // of buffer 0 are the first of buffer 1. The epilogue takes the shared columns first and
    // reports them read, and a tile's first instruction waits for that report of the tile
    // before it (and for the whole of the one before that, as without sharing).
    static constexpr int SFC = SFK * 4 * (1 + SFB_TILES);
    static constexpr int OV = FP4 && ACC_COLS == 256 ? 2 * SFC : 0;
    // groups of epilogue warps (of one column range, four lane quadrants) that hold shared columns
    static constexpr int OV_GROUPS = (OV + BN / (EW / 4) - 1) / (BN / (EW / 4));
    static constexpr int ACC0 = FP4 ? (OV ? OV : 128) : 0;
    static constexpr int ACC1 = FP4 ? (OV ? 256 : ACC0 + ACC_COLS) : ACC_COLS;
    static constexpr int TMEM_COLS = FP4 ? 512 : 2 * ACC_COLS;  // two accumulator buffers
    static_assert(!FP4 || (2 * SFC <= ACC0 && ACC1 + ACC_COLS <= 512), "columns of the scales");
    // DUAL: the W_g and W_u boxes form one 2*BN-row B tile (on one CTA, back to back; in a
    // pair, W_g on the leader and W_u on the peer), so one instruction fills gate columns
    // [0, BN) and up columns [BN, 2BN).
    static constexpr uint32_t IDESC =
        FP4 ? idesc_fp4(MMA_N, TILE_M, !NV) : idesc_mma(MMA_N, TILE_M, A_MN, B_MN, FP8);
    static_assert(!(FP8 || FP4) || (!A_MN && !B_MN && !WGRAD && !TWO_K),
                  "E4M3 and E2M1: K-major GEMMs");
    static_assert(TMEM_COLS == 256 || TMEM_COLS == 512, "tensor memory columns");
    static_assert(BN % 64 == 0 && MMA_N <= 256 && BROWS % (FP4 ? 32 : 64) == 0, "tile width");
    static constexpr size_t MISC_BYTES = 512 + sizeof(int64_t) * (kMaxExperts + 1) +
                                         (FP4 ? 0 : sizeof(int32_t) * kMaxExperts) +
                                         sizeof(int32_t) * (kMaxExperts + 1);
    static constexpr size_t SMEM_BYTES =
        1024 + (size_t)STAGES * STAGE_BYTES + AU_BYTES + OUT_BYTES + CS_BYTES + MISC_BYTES;
    static_assert((3 * STAGES + 7 + EW * kAuBufs) * 8 + 8 <= 512, "barrier block");
    static_assert(!(OV && AU), "the SwiGLU backward reports no shared columns");
    static_assert(STAGES * SF_BYTES % 1024 == 0, "alignment of what follows the stages");

};

struct Params {
    const int64_t* row_offsets;  // padded expert segments, or null = one dense expert
    const int32_t* expert_order; // weight gradients: experts in descending row count
    int64_t rows;                // extent of the token dimension
    int E;
    int N;      // output columns
    int K0;     // token-major: reduction length of operand pair 0
    int K1;     // token-major: reduction length of operand pair 1 (TWO_K)
    int M_out;  // weight gradients: rows of each expert's output
    int nprob;  // weight gradients: (a0,out0) and, if 2, (a1,out1)
    int kb_per_expert;  // B operand rows per expert (MN-major weights: K extent per expert)
    // weight gradients: the outputs of problems 0 and 1 (token-major outputs leave through
    // the output tensor maps instead)
    __nv_bfloat16* out0;
    __nv_bfloat16* out1;
    const float* sa;           // FP8: scale of each A row (indexed by the global row)
    const float* sb0;          // FP8: scale of each B row (output channel), first B operand
    const float* sb1;          // FP8: second B operand (W_u of G1)
    const float* row_scale;    // gate folded into the expert: G1 writes g*h, B2 forms g*dh
    float* gate_part;          // B2 with row_scale: per row, (dy W_d) . h per 64 columns
    int ld_out;                // B2: output columns; gate_part holds ld_out / 64 per row
    // B4 with the router's input-gradient term in the rows: row += r1_row[row] * r1_col[e][col]
    // (the slot's logit gradient times its expert's router row, both fp32)
    const float* r1_row;
    const float* r1_col;
    bool only_h;               // E2M1 G1: h alone is written (nothing is kept for a backward)
    // MX: the operand of the bf16 outputs, formed from them in the epilogue (G1: of h; B2: of
    // [dA | dU]): codes and scale tiles, or null
    uint8_t* oq;
    uint8_t* os;
    int* status;
    uint64_t wait_limit_ns;
};

struct TileInfo {
    int e;       // expert
    int p;       // weight-gradient problem (0 or 1)
    int64_t m0;  // token-major: first row; weight gradients: first output row
    int n0;      // first output column
    int64_t k_lo;  // weight gradients: first token row of the expert
    int k_iters;   // 64-wide K blocks
    int64_t row_end;  // token-major: rows at or past this are not stored
};

struct SmemLayout {
    uint8_t* a;        // STAGES x A tile
    uint8_t* b;        // STAGES x B tile(s)
    uint8_t* sf;       // STAGES x scale tiles (E2M1): A's, then B's
    uint64_t* full;    // STAGES
    uint64_t* empty;   // STAGES
    uint64_t* tfull;   // 2
    uint64_t* tempty;  // 2
    uint64_t* sffull;  // STAGES: a stage's scales are in shared memory (E2M1)
    uint64_t* sfready; // 2: they are in tensor memory
    uint64_t* tshared; // the accumulators' shared columns are read (E2M1)
    uint32_t* tmem_slot;
    int* abort_flag;
    int64_t* offs;     // E + 1
    int32_t* order;    // E
    int32_t* ptp;      // E + 1: exclusive prefix of pair tiles per expert (pair, token-major)
    uint8_t* au;       // SwiGLU backward: EW x kAuBufs staged (a | u) chunks
    uint64_t* au_full; // EW x kAuBufs
    float* cs;         // NV: EW x CS_FLOATS columns' powers of two
    uint8_t* ob;       // TMA-store epilogues: EW x OUT_DEPTH staged output chunks
};

template <class C>
__device__ __forceinline__ SmemLayout carve(uint8_t* raw) {
    SmemLayout s;
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    s.a = base;
    s.b = base + (size_t)C::STAGES * C::A_BYTES;
    s.sf = base + (size_t)C::STAGES * (C::A_BYTES + C::B_BYTES);
    s.au = base + (size_t)C::STAGES * C::STAGE_BYTES;  // 1024-aligned: the stages are together
    s.ob = s.au + C::AU_BYTES;  // 1024-aligned: the a/u buffers are whole KB
    s.cs = reinterpret_cast<float*>(s.ob + C::OUT_BYTES);
    uint8_t* misc = s.ob + C::OUT_BYTES + C::CS_BYTES;
    s.full = reinterpret_cast<uint64_t*>(misc);
    s.empty = s.full + C::STAGES;
    s.tfull = s.empty + C::STAGES;
    s.tempty = s.tfull + 2;
    s.tshared = s.tempty + 2;
    s.sffull = s.tshared + 1;
    s.sfready = s.sffull + C::STAGES;
    s.au_full = s.sfready + 2;
    s.tmem_slot = reinterpret_cast<uint32_t*>(s.au_full + (C::AU ? C::EW * kAuBufs : 0));
    s.abort_flag = reinterpret_cast<int*>(s.tmem_slot + 1);
    s.offs = reinterpret_cast<int64_t*>(misc + 512);
    s.order = reinterpret_cast<int32_t*>(s.offs + kMaxExperts + 1);
    s.ptp = s.order + (C::FP4 ? 0 : kMaxExperts);
    return s;
}

__device__ __forceinline__ int64_t cdiv_dev(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles along N; E2M1's last one may reach past it (its operands there are other rows or zeros, its
// outputs are clipped by the stores).
template <class C>
__device__ __forceinline__ int col_tiles(const Params& P) {
    return C::FP4 ? (P.N + C::BN - 1) / C::BN : P.N / C::BN;
}

template <class C>
__device__ __forceinline__ int64_t total_tiles(const Params& P, const SmemLayout& S) {
    const int n_tiles = col_tiles<C>(P);
    if constexpr (C::WGRAD) {
        return (int64_t)P.E * P.nprob * (P.M_out / C::TILE_M) * n_tiles;
    } else {
        int64_t mt;
        if (!P.row_offsets) mt = cdiv_dev(P.rows, C::TILE_M);
        else if (C::PAIR) mt = S.ptp[P.E];
        else mt = S.offs[P.E] / BM;
        return mt * n_tiles;
    }
}

// Last expert e in [0, E) with key[e] <= v (key non-decreasing). Among equal keys (empty
// experts) the last one is the expert that owns the rows.
template <class K>
__device__ __forceinline__ int last_le(const K* key, int E, int64_t v) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)key[mid] <= v) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Tile `tile` as seen by CTA `rank` of its pair (rank 0 outside pair mode).
template <class C>
__device__ __forceinline__ TileInfo decode(int64_t tile, const Params& P, const SmemLayout& S,
                                           uint32_t rank) {
    TileInfo ti;
    const int n_tiles = col_tiles<C>(P);
    const int64_t half = C::PAIR ? (int64_t)rank * BM : 0;
    if constexpr (C::WGRAD) {
        const int m_tiles = P.M_out / C::TILE_M;
        const int64_t per_e = (int64_t)P.nprob * m_tiles * n_tiles;
        const int oi = (int)(tile / per_e);
        int64_t rem = tile % per_e;
        ti.e = S.order[oi];
        ti.p = (int)(rem / (m_tiles * n_tiles));
        rem %= (m_tiles * n_tiles);
        ti.m0 = (rem / n_tiles) * C::TILE_M + half;
        ti.n0 = (int)(rem % n_tiles) * C::BN;
        int64_t lo = 0, hi = P.rows;
        if (P.row_offsets) {
            lo = S.offs[ti.e];
            hi = S.offs[ti.e + 1];
        }
        ti.k_lo = lo;
        ti.k_iters = (int)cdiv_dev(hi - lo, BK);
        ti.row_end = P.M_out;
    } else {
        const int64_t mt = tile / n_tiles;
        ti.n0 = (int)(tile % n_tiles) * C::BN;
        ti.p = 0;
        ti.k_lo = 0;
        ti.e = 0;
        if (!P.row_offsets) {
            ti.m0 = mt * C::TILE_M + half;
            ti.row_end = P.rows;
        } else if constexpr (C::PAIR) {
            // pair tiles of expert e cover its padded segment 256 rows at a time; the
            // second half of a segment's last pair tile may lie past the segment
            ti.e = last_le(S.ptp, P.E, mt);
            ti.m0 = S.offs[ti.e] + (mt - S.ptp[ti.e]) * C::TILE_M + half;
            ti.row_end = S.offs[ti.e + 1];
        } else {
            ti.m0 = mt * BM;
            ti.e = last_le(S.offs, P.E, ti.m0);
            ti.row_end = S.offs[ti.e + 1];
        }
        ti.k_iters = (P.K0 + (C::TWO_K ? P.K1 : 0)) / C::KB;
    }
    return ti;
}

// The same for E2M1, whose tiles take as long as decode's 64-bit divisions and search: 32-bit
// arithmetic (the launch has fewer than 2^31 tiles), and the expert found from the last tile's, as
// the tiles a CTA takes ascend. The MMA and copying threads need no more of a tile than its columns.
template <class C>
__device__ __forceinline__ TileInfo decode_fp4(uint32_t tile, int& e, const Params& P,
                                               const SmemLayout& S, uint32_t rank) {
    TileInfo ti;
    const uint32_t n_tiles = col_tiles<C>(P);
    const uint32_t mt = tile / n_tiles;
    ti.n0 = (int)(tile - mt * n_tiles) * C::BN;
    ti.p = 0;
    ti.k_lo = 0;
    ti.k_iters = (P.K0 + C::KB - 1) / C::KB;  // the last may be half a block
    const int64_t half = C::PAIR ? (int64_t)rank * BM : 0;
    if (!P.row_offsets) {
        ti.e = 0;
        ti.m0 = (int64_t)mt * C::TILE_M + half;
        ti.row_end = P.rows;
    } else if constexpr (C::PAIR) {
        while (e + 1 < P.E && (uint32_t)S.ptp[e + 1] <= mt) ++e;
        ti.e = e;
        ti.m0 = S.offs[e] + (int64_t)(mt - S.ptp[e]) * C::TILE_M + half;
        ti.row_end = S.offs[e + 1];
    } else {
        ti.m0 = (int64_t)mt * BM;
        while (e + 1 < P.E && S.offs[e + 1] <= ti.m0) ++e;
        ti.e = e;
        ti.row_end = S.offs[e + 1];
    }
    return ti;
}

template <class C>
__device__ __forceinline__ TileInfo next_tile(int64_t tile, int& e, const Params& P,
                                              const SmemLayout& S, uint32_t rank) {
    if constexpr (C::FP4) return decode_fp4<C>((uint32_t)tile, e, P, S, rank);
    else return decode<C>(tile, P, S, rank);
}

template <class C>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                         int32_t c0, int32_t c1) {
    if constexpr (C::PAIR) tma_load_2d_pair(dst, map, bar, c0, c1);
    else tma_load_2d(dst, map, bar, c0, c1);
}

// Loads of K block `kb` of an E2M1 tile. Where K ends inside the block (K is a multiple of 128)
// the codes past it read as zero and the scales past it are whatever lies there; no
// instruction uses either.
template <class C>
__device__ __forceinline__ void issue_loads_fp4(const TileInfo& ti, int kb, uint32_t a_dst,
                                                uint32_t b_dst, uint32_t sf_dst, uint32_t bar,
                                                uint32_t sf_bar, const Params& P, const CUtensorMap* ma0,
                                                const CUtensorMap* mb0, const CUtensorMap* mb1,
                                                const CUtensorMap* msa, const CUtensorMap* msb0,
                                                const CUtensorMap* msb1, uint32_t rank) {
    const int32_t kbyte = kb * (C::KB / 2);
    const int32_t ktiles = P.K0 / (C::KB / C::SFK);  // scale tiles along K
    const int32_t kt = kb * C::SFK;
    const int32_t brow = ti.e * P.N + ti.n0;  // N is a multiple of 128, n0 at least of 64
    // the scales first: they are copied on while the operands still arrive
    tma_load<C>(sf_dst, msa, sf_bar, 0, (int32_t)(ti.m0 / BM) * ktiles + kt);
#pragma unroll
    for (int h = 0; h < C::SFB_TILES; ++h)
        tma_load<C>(sf_dst + (1 + h) * C::SFA_BYTES, C::DUAL && h == 1 ? msb1 : msb0, sf_bar, 0,
                    (brow / BM + (C::DUAL ? 0 : h)) * ktiles + kt);
    tma_load<C>(a_dst, ma0, bar, kbyte, (int32_t)ti.m0);
    if constexpr (C::DUAL) {
        if constexpr (C::PAIR) {
            tma_load<C>(b_dst, rank == 0 ? mb0 : mb1, bar, kbyte, brow);
        } else {
            tma_load<C>(b_dst, mb0, bar, kbyte, brow);
            tma_load<C>(b_dst + C::BN * 128, mb1, bar, kbyte, brow);
        }
    } else {
        tma_load<C>(b_dst, mb0, bar, kbyte, brow + (C::PAIR ? (int32_t)rank * C::BROWS : 0));
    }
}

// The scales of one E2M1 K block of `steps` steps of 64 into tensor memory (column tmem_sf on): tiles
// `half` * SFK / 2 on, half of them; the other copying thread takes the rest. sf_lo: low word of the
// descriptor of the stage's first scale tile.
template <class C>
__device__ __forceinline__ void issue_scales_fp4(uint32_t tmem_sf, uint32_t sf_lo, int steps, int half) {
    const uint32_t sfb = tmem_sf + C::SFK * 4;
    const int tiles = C::NV ? steps : steps / 2;
#pragma unroll
    for (int i = 0; i < C::SFK / 2; ++i) {
        const int t = half * (C::SFK / 2) + i;
        if (t >= tiles) break;
        tmem_cp_scales<C::PAIR>(tmem_sf + 4 * t, sf_lo + t * (kSfTile / 16));
#pragma unroll
        for (int h = 0; h < C::SFB_TILES; ++h)
            tmem_cp_scales<C::PAIR>(sfb + 4 * (C::SFB_TILES * t + h),
                                    sf_lo + ((1 + h) * C::SFA_BYTES + t * kSfTile) / 16);
    }
}

// One step of 64 K elements of an E2M1 K block; a_lo and b_lo: low words of the descriptors of the
// stage's operands, sfb: column of the B scales.
template <class C, int KK>
__device__ __forceinline__ void issue_step_fp4(uint32_t d_tmem, uint32_t sfa, uint32_t sfb,
                                               uint32_t a_lo, uint32_t b_lo, uint32_t accumulate) {
    constexpr int t = C::NV ? KK : KK / 2;
    constexpr uint32_t id = C::NV ? 0u : 2u * (KK & 1);  // which half of the tile's four blocks
    umma_fp4<C::PAIR, C::NV>(d_tmem, a_lo + 2 * KK, b_lo + 2 * KK, C::IDESC | (id << 29) | (id << 4),
                             sfa + 4 * t, sfb + 4 * C::SFB_TILES * t, accumulate);
}

// Loads of K block `kb` of a tile into this CTA's stage buffers; `bar` is the barrier the
// copies complete on (in pair mode the leader's, as a shared::cluster address).
template <class C>
__device__ __forceinline__ void issue_loads(const TileInfo& ti, int kb, uint32_t a_dst,
                                            uint32_t b_dst, uint32_t bar, const Params& P,
                                            const CUtensorMap* ma0, const CUtensorMap* ma1,
                                            const CUtensorMap* mb0, const CUtensorMap* mb1,
                                            uint32_t rank) {
    const int32_t bhalf = C::PAIR ? (int32_t)rank * C::BROWS : 0;  // this CTA's B columns
    if constexpr (C::WGRAD) {
        const int32_t krow = (int32_t)(ti.k_lo + (int64_t)kb * BK);
        const CUtensorMap* ma = ti.p == 0 ? ma0 : ma1;
        // A: MN-major, two 64-wide boxes along M
        tma_load<C>(a_dst, ma, bar, (int32_t)ti.m0, krow);
        tma_load<C>(a_dst + 8192, ma, bar, (int32_t)ti.m0 + 64, krow);
#pragma unroll
        for (int j = 0; j < C::BROWS / 64; ++j)
            tma_load<C>(b_dst + j * 8192, mb0, bar, ti.n0 + bhalf + 64 * j, krow);
    } else {
        int kk = kb * C::KB;
        const CUtensorMap* ma = ma0;
        const CUtensorMap* mb = mb0;
        int kper = P.kb_per_expert;
        if (C::TWO_K && kk >= P.K0) {
            kk -= P.K0;
            ma = ma1;
            mb = mb1;
        }
        tma_load<C>(a_dst, ma, bar, kk, (int32_t)ti.m0);
        if constexpr (C::B_MN) {
            const int32_t brow = ti.e * kper + kk;
#pragma unroll
            for (int j = 0; j < C::BROWS / 64; ++j)
                tma_load<C>(b_dst + j * 8192, mb, bar, ti.n0 + bhalf + 64 * j, brow);
        } else if constexpr (C::DUAL) {
            const int32_t brow = ti.e * P.N + ti.n0;
            if constexpr (C::PAIR) {
                tma_load<C>(b_dst, rank == 0 ? mb0 : mb1, bar, kk, brow);
            } else {
                tma_load<C>(b_dst, mb0, bar, kk, brow);
                tma_load<C>(b_dst + C::BN * 128, mb1, bar, kk, brow);
            }
        } else {
            tma_load<C>(b_dst, mb, bar, kk, ti.e * P.N + ti.n0 + bhalf);
        }
    }
}

__device__ __forceinline__ uint4 pack_chunk8(const float* v) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}

// FP8 dequantisation of a 32-column accumulator chunk: value * scale(A row) * scale(B row
// of each output column). With dual=true, `a` takes the first B operand's column scales
// and `b` the second's (G1: gate and up); otherwise only `a` is scaled.
template <int W = 32>
__device__ __forceinline__ void fp8_scale(float* a, float* b, const Params& P, int64_t row,
                                          const TileInfo& ti, int c, bool dual = true) {
    const float sr = __ldg(P.sa + row);
    const int64_t col0 = (int64_t)ti.e * P.N + ti.n0 + c;
    const float4* s0 = reinterpret_cast<const float4*>(P.sb0 + col0);
#pragma unroll
    for (int q = 0; q < W / 4; ++q) {
        const float4 v = __ldg(s0 + q);
        a[4 * q] *= sr * v.x;
        a[4 * q + 1] *= sr * v.y;
        a[4 * q + 2] *= sr * v.z;
        a[4 * q + 3] *= sr * v.w;
    }
    if (dual) {
        const float4* s1 = reinterpret_cast<const float4*>(P.sb1 + col0);
#pragma unroll
        for (int q = 0; q < W / 4; ++q) {
            const float4 v = __ldg(s1 + q);
            b[4 * q] *= sr * v.x;
            b[4 * q + 1] *= sr * v.y;
            b[4 * q + 2] *= sr * v.z;
            b[4 * q + 3] *= sr * v.w;
        }
    }
}

// The slot's router term in a chunk of a data-gradient row, one fp32 FMA per element.
template <int W>
__device__ __forceinline__ void add_router_term(float* v, const Params& P, int64_t row,
                                                const TileInfo& ti, int c) {
    const float g = __ldg(P.r1_row + row);
    const float4* w =
        reinterpret_cast<const float4*>(P.r1_col + (int64_t)ti.e * P.N + ti.n0 + c);
#pragma unroll
    for (int j = 0; j < W / 4; ++j) {
        const float4 w4 = __ldg(w + j);
        v[4 * j] = fmaf(g, w4.x, v[4 * j]);
        v[4 * j + 1] = fmaf(g, w4.y, v[4 * j + 1]);
        v[4 * j + 2] = fmaf(g, w4.z, v[4 * j + 2]);
        v[4 * j + 3] = fmaf(g, w4.w, v[4 * j + 3]);
    }
}

// Weight-gradient epilogue: columns [c_lo, c_hi) of this thread's output row (a weight row;
// always inside the output, as M_out and N are whole tiles). An expert with no rows gives
// zeros.
template <class C>
__device__ __forceinline__ void epilogue_wgrad(const TileInfo& ti, uint32_t t_acc, int row_in_tile,
                                               const Params& P, int c_lo, int c_hi) {
    static_assert(C::WGRAD, "weight-gradient tiles only");
    const int64_t row = ti.m0 + row_in_tile;
    __nv_bfloat16* out = (ti.p == 0 ? P.out0 : P.out1) + ((int64_t)ti.e * P.M_out + row) * P.N + ti.n0;
    for (int c = c_lo; c < c_hi; c += 32) {
        float v[32];
        if (ti.k_iters > 0) {
            uint32_t r[32];
            tmem_ld32(t_acc + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.f;
        }
        uint4* dst = reinterpret_cast<uint4*>(out + c);
#pragma unroll
        for (int q = 0; q < 4; ++q) dst[q] = pack_chunk8(v + 8 * q);
    }
}

// ------------------------------------------------------- epilogues with TMA stores
// Each epilogue warp owns 32 rows x (BN / 2) columns of the tile and walks them in chunks of
// kOutCols. Per chunk its lanes pack their rows of every output into a shared-memory buffer
// laid out as the 32-byte-swizzled TMA box (kOutCols x 32 rows), and lane 0 stores the boxes;
// a buffer is rewritten only after the store that read it two chunks earlier is done.
// A 128-row half of a pair tile that lies past the expert's segment stores nothing (such a
// half is wholly inside or wholly outside, as segments are padded to 128 rows); rows past
// the end of the output tensor are clipped by the stores themselves.

// Byte offset of 16-byte piece j of row r in a 32-byte-swizzled box of 32-byte rows.
__device__ __forceinline__ int sw32_offset(int r, int j) { return r * 32 + ((j ^ ((r >> 2) & 1)) << 4); }
// ... and in a 64-byte-swizzled box of 64-byte rows (32 bf16 columns).
__device__ __forceinline__ int sw64_offset(int r, int j) { return r * 64 + ((j ^ ((r >> 1) & 3)) << 4); }

template <int W>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[W]) {
    if constexpr (W == 32) tmem_ld32(taddr, r);
    else if constexpr (W == 16) tmem_ld16(taddr, r);
    else tmem_ld8(taddr, r);
}


template <class C>
__device__ __forceinline__ void epilogue_tma_store(const SmemLayout& S, const TileInfo& ti,
                                                   uint32_t t_acc, int q, int lane, int slot,
                                                   int c_lo, int ncols, const Params& P,
                                                   const CUtensorMap* mo0, const CUtensorMap* mo1,
                                                   const CUtensorMap* mo2, uint32_t& n) {
    constexpr int W = C::OCOLS;
    if (ti.m0 >= ti.row_end) return;  // warp-uniform: the whole half is past the segment
    const int64_t row0 = ti.m0 + 32 * q;
    // rows past row_end (the tail of an unpadded layout) are clipped by the store; their FP8
    // row scale is read from the last row instead
    const int64_t row = row0 + lane < ti.row_end ? row0 + lane : ti.row_end - 1;
    for (int i = 0; i < ncols / W; ++i, ++n) {
        const int c = c_lo + i * W;
        float v[C::NOUT][W];
        if constexpr (C::EPI == kEpiSwigluFwd) {
            uint32_t g[W], u[W];
            tmem_ld_cols<W>(t_acc + c, g);
            tmem_ld_cols<W>(t_acc + C::BN + c, u);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < W; ++j) {
                v[0][j] = __uint_as_float(g[j]);
                v[1][j] = __uint_as_float(u[j]);
            }
            if constexpr (C::FP8) fp8_scale<W>(v[0], v[1], P, row, ti, c);
            const float rg = P.row_scale ? __ldg(P.row_scale + row) : 1.0f;
#pragma unroll
            for (int j = 0; j < W; ++j)
                v[2][j] = v[0][j] / (1.0f + __expf(-v[0][j])) * v[1][j] * rg;
        } else {
            uint32_t r[W];
            tmem_ld_cols<W>(t_acc + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < W; ++j) v[0][j] = __uint_as_float(r[j]);
            if constexpr (C::FP8) fp8_scale<W>(v[0], v[0], P, row, ti, c, /*dual=*/false);
            if constexpr (C::EPI == kEpiStore && !C::WGRAD)
                if (P.r1_row) add_router_term<W>(v[0], P, row, ti, c);
        }
        uint8_t* buf = S.ob + ((size_t)slot * C::OUT_DEPTH + n % C::OUT_DEPTH) * C::OUT_BUF_BYTES;
        if (lane == 0) bulk_wait_read<C::OUT_DEPTH - 1>();  // the store that last read it is done
        __syncwarp();
#pragma unroll
        for (int o = 0; o < C::NOUT; ++o)
#pragma unroll
            for (int j = 0; j < W / 8; ++j)
                *reinterpret_cast<uint4*>(buf + o * C::OUT_BOX_BYTES +
                                          (W == 32 ? sw64_offset(lane, j) : sw32_offset(lane, j))) =
                    pack_chunk8(v[o] + 8 * j);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            const CUtensorMap* mo[3] = {mo0, mo1, mo2};
#pragma unroll
            for (int o = 0; o < C::NOUT; ++o)
                tma_store_2d(mo[o], smem_u32(buf + o * C::OUT_BOX_BYTES), ti.n0 + c, (int32_t)row0);
            bulk_commit();
        }
    }
}

// ------------------------------------------------- outputs of the E2M1 GEMMs
// A tile's main loop is a quarter of the bf16 one's, so the number of rows that the TMA stores
// move and the time from a tile's last instruction until its columns are free set the pace. Boxes are
// up to 64 columns x 32 rows, whole 128-byte lines (with 16-column boxes the gate and up projections
// of experts of 768 took 1144 us, with 64-column ones 540). Eight warps take 64 (gate and up) or 128
// columns each, twelve 64 of 192 columns; a warp reads its shared columns, or all of them where they
// fit in registers, before it packs any, so that the next tile's instructions wait for the loads only.

// Byte offset of 16-byte piece j of row r in a 128-byte-swizzled box of 128-byte rows.
__device__ __forceinline__ int sw128_offset(int r, int j) { return r * 128 + ((j ^ (r & 7)) << 4); }

// NV: the powers of two of a tile's columns (of each accumulator) on their way into this warp's place in
// shared memory; that of this thread's row is returned. They are asked for as soon as those of the tile
// before have been used: where a tile has few stages, its main loop would not cover their latency
// (8191 tokens through 8 of 64 experts of 1024 x 256: 107 us a pass, 109 with them fetched as a tile
// begins; 115 in its epilogue).
template <class C>
__device__ __forceinline__ float start_powers(float* cs, const Params& P, const TileInfo& ti, int row_in_tile,
                                              int c_lo, int lane) {
    constexpr int kCols = C::BN / (C::EW / 4);
    static_assert(C::CS_FLOATS <= 128, "one copy a lane");
    __syncwarp();  // the previous tile's have been used
    if (ti.m0 >= ti.row_end) return 1.0f;
    const int j = 4 * lane;  // of gate, then of up
    const int c = ti.n0 + c_lo + j % kCols;
    if (j < C::CS_FLOATS && c < P.N)
        cp_async16(cs + j, (C::DUAL && j >= kCols ? P.sb1 : P.sb0) + (int64_t)ti.e * P.N + c);
    const int64_t r = ti.m0 + row_in_tile;
    return __ldg(P.sa + (r < ti.row_end ? r : ti.row_end - 1));
}
// Then an accumulator chunk of 32 columns times both, as one number: exact, or scale_in_place has been there
// first and both are 1.
__device__ __forceinline__ void apply_powers(float* v, float g, const float* cs) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const float4 w = reinterpret_cast<const float4*>(cs)[q];
        v[4 * q] *= g * w.x;
        v[4 * q + 1] *= g * w.y;
        v[4 * q + 2] *= g * w.z;
        v[4 * q + 3] *= g * w.w;
    }
}

// A power is 2^-126 to 2^118, so that a row's times a column's can leave fp32's range where the scaled sum
// does not: sums of zeros would be NaN under 2^89 and 2^89, one of 2^30 would be 0 under 2^-102 and
// 2^-49. Whether this warp's all lie within 2^63 of 1, whose products are exact (the same for all lanes).
template <class C>
__device__ __forceinline__ bool powers_multiply(const float* cs, float g, int lane) {
    const float lo = 0x1p-63f, hi = 0x1p63f;
    bool ok = g >= lo && g <= hi;
    if (4 * lane < C::CS_FLOATS) {
        const float4 w = reinterpret_cast<const float4*>(cs)[lane];
        ok = ok && w.x >= lo && w.x <= hi && w.y >= lo && w.y <= hi && w.z >= lo && w.z <= hi &&
             w.w >= lo && w.w <= hi;
    }
    return __all_sync(0xffffffffu, ok);
}
// Where they do not, the tile's part of this warp (t_warp: its columns of the first accumulator) is scaled in
// tensor memory before its epilogue, 32 columns at a time, and ones take the place of the powers. Powers
// on different sides of 1 are multiplied first, which is exact; those on the same side one after the
// other, each taking the sum further the same way. Out of line, for the registers of the epilogues: 8191
// tokens through 8 of 64 experts of 1024 x 256 take 113 us a pass with the caches flushed (111 without the
// question), 115 with this inlined and 122 with the choice made among the accumulators that an epilogue holds.
template <class C>
__device__ __noinline__ void scale_in_place(uint32_t t_warp, float g, float* cs, int lane) {
    constexpr int kCols = C::BN / (C::EW / 4);
#pragma unroll 1
    for (int j = 0; j < C::CS_FLOATS; j += 32) {  // of gate, then of up
        const uint32_t at = t_warp + (C::DUAL && j >= kCols ? C::BN - kCols : 0) + j;
        uint32_t r[32];
        tmem_ld32(at, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float v = __uint_as_float(r[i]), w = cs[j + i];
            r[i] = __float_as_uint((g < 1.0f) == (w < 1.0f) ? v * g * w : v * (g * w));
        }
        tmem_st32(at, r);
    }
    tmem_st_wait();
    __syncwarp();  // every lane has used the powers
    if (4 * lane < C::CS_FLOATS) reinterpret_cast<float4*>(cs)[lane] = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    __syncwarp();
}

// 32 packed columns of this thread's row into its place in a box of C::OCOLS columns.
template <class C>
__device__ __forceinline__ void put_half(uint8_t* buf, int lane, int half, const uint32_t* w) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(buf + (C::OCOLS == 64 ? sw128_offset(lane, 4 * half + j)
                                                        : sw64_offset(lane, j))) =
            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}

// An MX block (32 packed columns from `col` on, of this thread's row) to its codes and its scale in an
// operand of `cols` columns, as quantising the stored bf16 row does. A warp writes half a sector of
// codes and a byte of a scale word a row; the second block of the two that a warp has fills both.
__device__ __forceinline__ void store_mx_block(const uint32_t (&w)[16], uint8_t* q, uint8_t* s, int cols,
                                               int64_t row, int col) {
    uint4 codes;
    const uint32_t byte = mx_block(w, codes);
    *reinterpret_cast<uint4*>(q + row * (cols / 2) + col / 2) = codes;
    s[fp4_scale_word(row, col / 128, cols / 128) + col % 128 / 32] = (uint8_t)byte;
}

// Arrivals at the leading CTA's barriers (this CTA's, outside pairs) that a warp's reads are over: of
// the columns shared with the next tile's accumulator, and of the whole one.
struct Readers {
    bool shared;            // this warp holds shared columns
    uint32_t shared_bar, whole_bar;
};
template <class C>
__device__ __forceinline__ void arrive_read(uint32_t bar, int lane) {
    tc_fence_before();
    __syncwarp();
    if (lane != 0) return;
    if constexpr (C::PAIR) mbar_arrive_cluster_relaxed(bar);
    else mbar_arrive(bar);
}

// next_powers(): called once the tile's powers of two have been used (NV).
template <class C, class Next>
__device__ __forceinline__ void epilogue_fp4(const SmemLayout& S, const TileInfo& ti, uint32_t t_acc,
                                             int lane, int slot, int c_lo, int64_t row0, const Params& P,
                                             const CUtensorMap* mo0, const CUtensorMap* mo1,
                                             const CUtensorMap* mo2, bool reversed, const Readers& rd,
                                             float g_row, const float* cs, const Next& next_powers) {
    constexpr int kCols = C::BN / (C::EW / 4);    // of this warp (in each accumulator)
    // nothing to write: the half of a pair's tile past its segment, columns past the outputs
    if (ti.m0 >= ti.row_end || (C::BN % 128 && ti.n0 + c_lo >= P.N)) {
        if (C::OV && rd.shared) arrive_read<C>(rd.shared_bar, lane);
        arrive_read<C>(rd.whole_bar, lane);
        next_powers();
        return;
    }
    // rows past row_end (the tail of an unpadded layout) are clipped by the store
    const int64_t row = row0 + lane < ti.row_end ? row0 + lane : ti.row_end - 1;
    uint8_t* buf = S.ob + (size_t)slot * C::OUT_DEPTH * C::OUT_BUF_BYTES;
    if constexpr (C::EPI == kEpiSwigluFwd) {
        constexpr int kHalves = C::OCOLS / 32;
        static_assert(kCols == C::OCOLS, "one box a warp and output");
        uint32_t g[kHalves][32], u[kHalves][32];
#pragma unroll
        for (int k = 0; k < kHalves; ++k) {
            tmem_ld32(t_acc + c_lo + 32 * k, g[k]);
            tmem_ld32(t_acc + C::BN + c_lo + 32 * k, u[k]);
        }
        tmem_ld_wait();
        if (C::OV && rd.shared) arrive_read<C>(rd.shared_bar, lane);
        arrive_read<C>(rd.whole_bar, lane);
        // An approximate quotient and exponential (2 ulp of fp32 each, ahead of the rounding of h to bf16): 7 in
        // a million of h are rounded to the other neighbour than with expf and a division, and few of their
        // codes move a step (the sums of y by 1e-4 of the whole; the error against 64 bits is the same 0.0017).
        // 32,768 tokens through 128 experts of 2048 x 768 take 638 us (MX), with expf and the quotient
        // corrected by its remainder 675, with expf and a division 1309.
        const float rg = P.row_scale ? __ldg(P.row_scale + row) : 1.0f;
        if constexpr (C::NV) {
#pragma unroll
            for (int k = 0; k < kHalves; ++k) {
                apply_powers(reinterpret_cast<float*>(g[k]), g_row, cs + 32 * k);
                apply_powers(reinterpret_cast<float*>(u[k]), g_row, cs + kCols + 32 * k);
            }
            next_powers();
        }
#pragma unroll
        for (int o = 0; o < 3; ++o) {  // a, u, h
            if (o < 2 && P.only_h) continue;
            uint8_t* box = buf + o % C::OUT_DEPTH * C::OUT_BUF_BYTES;
            if (lane == 0) bulk_wait_read<C::OUT_DEPTH - 1>();  // its last store has read it
            __syncwarp();
#pragma unroll
            for (int k = 0; k < kHalves; ++k) {
                const float* gf = reinterpret_cast<const float*>(g[k]);
                const float* uf = reinterpret_cast<const float*>(u[k]);
                uint32_t w[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float g0 = gf[2 * j], g1 = gf[2 * j + 1];
                    const float u0 = uf[2 * j], u1 = uf[2 * j + 1];
                    w[j] = o == 0   ? pack_bf16x2(g0, g1)
                           : o == 1 ? pack_bf16x2(u0, u1)
                                    : pack_bf16x2(__fdividef(g0, 1.0f + __expf(-g0)) * u0 * rg,
                                                  __fdividef(g1, 1.0f + __expf(-g1)) * u1 * rg);
                }
                put_half<C>(box, lane, k, w);
                if (!C::NV && o == 2 && P.oq && row0 + lane < ti.row_end)
                    store_mx_block(w, P.oq, P.os, P.N, row, ti.n0 + c_lo + 32 * k);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(o == 0 ? mo0 : o == 1 ? mo1 : mo2, smem_u32(box), ti.n0 + c_lo, (int32_t)row0);
                bulk_commit();
            }
        }
    } else {
        // halves of 32 columns in order, or (buffer 0 of accumulators that share columns) the last
        // first; those with shared columns are taken out of tensor memory at once
        constexpr int kHalves = kCols / 32;
        constexpr int kAhead = !C::OV || kHalves < (C::OV + 31) / 32 ? kHalves : (C::OV + 31) / 32;
        auto half = [&](int i) { return C::OV && reversed ? kHalves - 1 - i : i; };
        uint32_t r[kHalves][32];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) tmem_ld32(t_acc + c_lo + 32 * half(i), r[i]);
        tmem_ld_wait();
        if (C::OV && rd.shared) arrive_read<C>(rd.shared_bar, lane);
        if (kAhead == kHalves) arrive_read<C>(rd.whole_bar, lane);
#pragma unroll
        for (int i = 0; i < kHalves; ++i) {
            const int c = c_lo + 32 * half(i);
            if (i % 2 == 0) {
                if (i + 1 >= kAhead) {  // the rest of this box
#pragma unroll
                    for (int k = i < kAhead ? kAhead : i; k < i + 2; ++k)
                        tmem_ld32(t_acc + c_lo + 32 * half(k), r[k]);
                    tmem_ld_wait();
                    if (kAhead < kHalves && i + 2 == kHalves) arrive_read<C>(rd.whole_bar, lane);
                }
                // the store that last read this buffer is done
                if (lane == 0) bulk_wait_read<C::OUT_DEPTH - 1>();
                __syncwarp();
            }
            float* v = reinterpret_cast<float*>(r[i]);
            if constexpr (C::NV) {
                apply_powers(v, g_row, cs + c - c_lo);
                if (i == kHalves - 1) next_powers();
            }
            if (P.r1_row) add_router_term<32>(v, P, row, ti, c);
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
            uint8_t* box = buf + i / 2 % C::OUT_DEPTH * C::OUT_BUF_BYTES;
            put_half<C>(box, lane, half(i) & 1, w);
            if (i % 2 == 1) {
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(mo0, smem_u32(box), ti.n0 + (c & ~63), (int32_t)row0);
                    bulk_commit();
                }
            }
        }
    }
}

// ------------------------------------------------- SwiGLU backward with staged a and u
// Each epilogue warp owns 32 rows x (BN / 2) columns of the tile and walks them in chunks of
// kAuCols. The chunk's saved a and u arrive by TMA (boxes of kAuCols x 32 rows, swizzled
// so that the row-per-lane reads below hit distinct banks) into one of the warp's kAuBufs
// buffers; lane 0 issues the copy of chunk n + kAuBufs once the warp is done with chunk n,
// and a tile's first chunks before its accumulator is ready.

// Byte offset of 16-byte piece j of row r in a staged (a or u) chunk.
__device__ __forceinline__ int au_offset(int r, int j) {
    if constexpr (kAuCols == 32) return r * 64 + ((j ^ ((r >> 1) & 3)) << 4);  // 64-byte swizzle
    else if constexpr (kAuCols == 16) return r * 32 + ((j ^ ((r >> 2) & 1)) << 4);  // 32-byte
    else return r * 16;                                                            // unswizzled
}

template <class C>
__device__ __forceinline__ void au_issue(const SmemLayout& S, const CUtensorMap* ma,
                                         const CUtensorMap* mu, int slot, uint32_t n, int64_t row0,
                                         int col) {
    const int b = (int)(n % kAuBufs);
    const uint32_t dst = smem_u32(S.au + ((size_t)slot * kAuBufs + b) * C::AU_BUF_BYTES);
    const uint32_t bar = smem_u32(&S.au_full[slot * kAuBufs + b]);
    // relaxed: the buffer's previous contents were read into registers and used before the
    // warp synchronised, and the fill orders no earlier store of this thread; a releasing
    // arrive would wait for the warp's dA/dU stores to drain (measured: B2 1.7% slower)
    mbar_arrive_expect_tx_relaxed(bar, C::AU_BUF_BYTES);
    tma_load_2d(dst, ma, bar, col, (int32_t)row0);
    tma_load_2d(dst + C::AU_BUF_BYTES / 2, mu, bar, col, (int32_t)row0);
}

// One tile of this warp's columns [c_lo, c_lo + ncols). `n` counts the warp's chunks over the
// kernel's life (it picks buffer and phase). Returns false when a wait failed (uniform
// across the warp).
template <class C>
__device__ __forceinline__ bool swiglu_bwd_staged(const SmemLayout& S, const TileInfo& ti,
                                                  uint32_t t_acc, int q, int lane, int slot,
                                                  int c_lo, int ncols, const Params& P,
                                                  const CUtensorMap* ma, const CUtensorMap* mu,
                                                  const CUtensorMap* mda, const CUtensorMap* mdu,
                                                  uint32_t& n, volatile int* abort_flag) {
    static_assert(kAuCols == kOutCols, "one staged output chunk per a/u chunk");
    const int nch = ncols / kAuCols;
    const int64_t row0 = ti.m0 + 32 * q;
    const int64_t row = row0 + lane;
    const bool ok_row = row < ti.row_end;
    // padded segments are whole 128-row halves, so a warp's rows are all inside or all past
    // the segment; rows past an unpadded layout's end are clipped by the store
    const bool store = row0 < ti.row_end;
    // gate folded into the expert: dy is the ungated row gradient, dh = g (dy W_d), and the
    // gate's gradient (dy W_d) . h is summed per 64-column group (h recomputed in fp32)
    const float g = (P.row_scale && ok_row) ? __ldg(P.row_scale + row) : 1.0f;
    float gpart = 0.f;
    for (int i = 0; i < nch; ++i, ++n) {
        const int c = c_lo + i * kAuCols;
        const int b = (int)(n % kAuBufs);
        uint32_t acc[kAuCols];
        tmem_ld_cols<kAuCols>(t_acc + c, acc);
        bool ok = mbar_wait_bounded(smem_u32(&S.au_full[slot * kAuBufs + b]), (n / kAuBufs) & 1u,
                                    abort_flag, P.status, P.wait_limit_ns, 34);
        tmem_ld_wait();
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
        float dav[kAuCols], duv[kAuCols];
        if (store) {  // lanes past an unpadded layout's end see zero-filled a, u and acc
            const uint8_t* abuf = S.au + ((size_t)slot * kAuBufs + b) * C::AU_BUF_BYTES;
            const uint8_t* ubuf = abuf + C::AU_BUF_BYTES / 2;
            float accf[kAuCols];
#pragma unroll
            for (int j = 0; j < kAuCols; ++j) accf[j] = __uint_as_float(acc[j]);
            // FP8 operands: the dequantised r = (dy codes) (W_d codes) * scale(row) * scale(col)
            if constexpr (C::FP8)
                fp8_scale<kAuCols>(accf, accf, P, ok_row ? row : ti.row_end - 1, ti, c, false);
#pragma unroll
            for (int j = 0; j < kAuCols / 8; ++j) {
                const uint4 a4 = *reinterpret_cast<const uint4*>(abuf + au_offset(lane, j));
                const uint4 u4 = *reinterpret_cast<const uint4*>(ubuf + au_offset(lane, j));
                const uint32_t aw[4] = {a4.x, a4.y, a4.z, a4.w};
                const uint32_t uw[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    const float a = (h & 1) ? bf16_hi(aw[h >> 1]) : bf16_lo(aw[h >> 1]);
                    const float u = (h & 1) ? bf16_hi(uw[h >> 1]) : bf16_lo(uw[h >> 1]);
                    const float acc_h = accf[8 * j + h];
                    const float sa = 1.0f / (1.0f + __expf(-a));
                    if (P.gate_part) gpart = fmaf(acc_h, a * sa * u, gpart);
                    const float dh = acc_h * g;
                    dav[8 * j + h] = dh * u * sa * (1.0f + a * (1.0f - sa));
                    duv[8 * j + h] = dh * a * sa;
                }
            }
            const int col = ti.n0 + c;
            if (P.gate_part && (col + kAuCols) % 64 == 0) {  // last chunk of a 64-column group
                if (ok_row) P.gate_part[row * (int64_t)(P.ld_out / 64) + col / 64] = gpart;
                gpart = 0.f;
            }
        }
        __syncwarp();  // every lane is done with a/u buffer b
        if (lane == 0 && i + kAuBufs < nch)
            au_issue<C>(S, ma, mu, slot, n + kAuBufs, row0, ti.n0 + c + kAuBufs * kAuCols);
        if (store) {
            uint8_t* ob = S.ob + ((size_t)slot * C::OUT_DEPTH + n % C::OUT_DEPTH) * C::OUT_BUF_BYTES;
            if (lane == 0) bulk_wait_read<C::OUT_DEPTH - 1>();  // the store that last read it is done
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kAuCols / 8; ++j) {
                *reinterpret_cast<uint4*>(ob + sw32_offset(lane, j)) = pack_chunk8(dav + 8 * j);
                *reinterpret_cast<uint4*>(ob + 1024 + sw32_offset(lane, j)) = pack_chunk8(duv + 8 * j);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(mda, smem_u32(ob), ti.n0 + c, (int32_t)row0);
                tma_store_2d(mdu, smem_u32(ob + 1024), ti.n0 + c, (int32_t)row0);
                bulk_commit();
            }
        }
    }
    return true;
}

// The same for E2M1, in 32-column chunks: a warp has 64 columns of a tile, so a tile's two chunks are
// staged whole while its main loop runs; dA and dU take the places of a and u in shared memory and
// leave from there. (In 16-column chunks with an output buffer beside them, and the correctly rounded
// quotient, the epilogue set the pace: 632 us with experts of 768, against 703 before that.)
template <class C>
__device__ __forceinline__ void au_issue_fp4(const SmemLayout& S, const CUtensorMap* ma,
                                             const CUtensorMap* mu, int slot, int64_t row0, int col) {
    bulk_wait_read<0>();  // the previous tile's dA and dU have left
#pragma unroll
    for (int b = 0; b < kAuBufs; ++b) {
        const uint32_t dst = smem_u32(S.au + ((size_t)slot * kAuBufs + b) * C::AU_BUF_BYTES);
        const uint32_t bar = smem_u32(&S.au_full[slot * kAuBufs + b]);
        mbar_arrive_expect_tx_relaxed(bar, C::AU_BUF_BYTES);
        tma_load_2d(dst, ma, bar, col + b * C::AUC, (int32_t)row0);
        tma_load_2d(dst + C::AU_BUF_BYTES / 2, mu, bar, col + b * C::AUC, (int32_t)row0);
    }
}

template <class C, class Next>
__device__ __forceinline__ bool swiglu_bwd_fp4(const SmemLayout& S, const TileInfo& ti,
                                               uint32_t t_acc, int q, int lane, int slot, int c_lo,
                                               const Params& P, const CUtensorMap* mda,
                                               const CUtensorMap* mdu, uint32_t local,
                                               volatile int* abort_flag, float g_row, const float* cs,
                                               const Next& next_powers) {
    const int64_t row0 = ti.m0 + 32 * q;
    const int64_t row = row0 + lane < ti.row_end ? row0 + lane : ti.row_end - 1;
    const bool store = row0 < ti.row_end;  // as in swiglu_bwd_staged
    bool ok = true;
#pragma unroll
    for (int b = 0; b < kAuBufs; ++b) {
        const int c = c_lo + b * C::AUC;
        uint32_t acc[32];
        tmem_ld32(t_acc + c, acc);
        ok = mbar_wait_bounded(smem_u32(&S.au_full[slot * kAuBufs + b]), local & 1u, abort_flag,
                               P.status, P.wait_limit_ns, 34) && ok;
        tmem_ld_wait();
        if (!__all_sync(0xffffffffu, ok)) return false;
        const bool in = store && ti.n0 + c < P.N;  // warp-uniform; N may end inside the last tile
        if (C::NV && in) apply_powers(reinterpret_cast<float*>(acc), g_row, cs + c - c_lo);
        if (C::NV && b == kAuBufs - 1) next_powers();
        if (!in) continue;
        uint8_t* abuf = S.au + ((size_t)slot * kAuBufs + b) * C::AU_BUF_BYTES;
        uint8_t* ubuf = abuf + C::AU_BUF_BYTES / 2;
        float* r = reinterpret_cast<float*>(acc);
        uint32_t wa[16], wu[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4* ap = reinterpret_cast<uint4*>(abuf + sw64_offset(lane, j));
            uint4* up = reinterpret_cast<uint4*>(ubuf + sw64_offset(lane, j));
            const uint4 a4 = *ap, u4 = *up;
            const uint32_t aw[4] = {a4.x, a4.y, a4.z, a4.w};
            const uint32_t uw[4] = {u4.x, u4.y, u4.z, u4.w};
            float da[8], du[8];
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                const float av = (h & 1) ? bf16_hi(aw[h >> 1]) : bf16_lo(aw[h >> 1]);
                const float uv = (h & 1) ? bf16_hi(uw[h >> 1]) : bf16_lo(uw[h >> 1]);
                // an approximate quotient (2 ulp); the correctly rounded one: 632 instead of 401 us
                // (before the codes of dA and dU were formed here; 458 with them)
                const float sa = __fdividef(1.0f, 1.0f + __expf(-av));
                const float dh = r[8 * j + h];
                da[h] = dh * uv * sa * (1.0f + av * (1.0f - sa));
                du[h] = dh * av * sa;
            }
            const uint4 pa = pack_chunk8(da), pu = pack_chunk8(du);
            *ap = pa;
            *up = pu;
            wa[4 * j] = pa.x, wa[4 * j + 1] = pa.y, wa[4 * j + 2] = pa.z, wa[4 * j + 3] = pa.w;
            wu[4 * j] = pu.x, wu[4 * j + 1] = pu.y, wu[4 * j + 2] = pu.z, wu[4 * j + 3] = pu.w;
        }
        if (!C::NV && P.oq && row0 + lane < ti.row_end) {  // the halves of [dA | dU]
            store_mx_block(wa, P.oq, P.os, 2 * P.N, row, ti.n0 + c);
            store_mx_block(wu, P.oq, P.os, 2 * P.N, row, P.N + ti.n0 + c);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(mda, smem_u32(abuf), ti.n0 + c, (int32_t)row0);
            tma_store_2d(mdu, smem_u32(ubuf), ti.n0 + c, (int32_t)row0);
            bulk_commit();
        }
    }
    return true;
}

// msa, msb0, msb1: scale tiles of A, the first and the second B operand (E2M1 only).
template <class C>
__device__ __forceinline__ void grouped_gemm_body(
    const CUtensorMap& ma0, const CUtensorMap& ma1, const CUtensorMap& mb0, const CUtensorMap& mb1,
    const CUtensorMap& mo0, const CUtensorMap& mo1, const CUtensorMap& mo2, const CUtensorMap* msa,
    const CUtensorMap* msb0, const CUtensorMap* msb1, const Params& P) {
    extern __shared__ uint8_t gg_smem_raw[];
    const SmemLayout S = carve<C>(gg_smem_raw);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t rank = C::PAIR ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    // tiles are dealt to CTAs (or to pairs, whose two CTAs take the same tile)
    const int64_t first_tile = C::PAIR ? blockIdx.x / 2 : blockIdx.x;
    const int64_t tile_step = C::PAIR ? gridDim.x / 2 : gridDim.x;

    if (tid == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&S.full[s]), 1);
            mbar_init(smem_u32(&S.empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&S.tfull[b]), 1);
            mbar_init(smem_u32(&S.tempty[b]), C::PAIR ? 2 * C::EW : C::EW);
        }
        if constexpr (C::OV > 0)
            mbar_init(smem_u32(S.tshared), 4 * C::OV_GROUPS * (C::PAIR ? 2 : 1));
        if constexpr (C::FP4) {
            for (int s = 0; s < C::STAGES; ++s) mbar_init(smem_u32(&S.sffull[s]), 1);
            for (int b = 0; b < 2; ++b) mbar_init(smem_u32(&S.sfready[b]), 2);  // both copying threads
        }
        if constexpr (C::AU)
            for (int b = 0; b < C::EW * kAuBufs; ++b) mbar_init(smem_u32(&S.au_full[b]), 1);
        *S.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 2) {
        if constexpr (C::PAIR) {
            tmem_alloc_pair(smem_u32(S.tmem_slot), C::TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(S.tmem_slot), C::TMEM_COLS);
            tmem_relinquish();
        }
    }
    if constexpr (C::FP4) {
        // Launched behind its stream's previous kernel: what is not read from memory that one writes
        // comes first. It does not let the next kernel start before it ends: one that did made the
        // chains of large GEMMs slower (data gradients of 128 experts 1037 instead of 1003 us).
        if (warp == 0 && lane == 0) {
            tma_prefetch_desc(&ma0);
            tma_prefetch_desc(&mb0);
            if (C::DUAL) tma_prefetch_desc(&mb1);
            tma_prefetch_desc(msa);
            tma_prefetch_desc(msb0);
            if (C::DUAL) tma_prefetch_desc(msb1);
        }
        __syncwarp();
        if constexpr (C::PAIR) cluster_sync();  // the peer's barriers exist before any remote use
        grid_dependency_wait();
    }
    if (P.row_offsets)
        for (int i = tid; i <= P.E; i += C::THREADS) S.offs[i] = P.row_offsets[i];
    if (C::WGRAD)
        for (int i = tid; i < P.E; i += C::THREADS) S.order[i] = P.expert_order ? P.expert_order[i] : i;
    if constexpr (C::PAIR && !C::WGRAD) {
        // pair tiles per expert = ceil(128-row tiles / 2); exclusive prefix in S.ptp
        __syncthreads();
        if (P.row_offsets) {
            int v = 0;
            if (tid < P.E) v = (int)(((S.offs[tid + 1] - S.offs[tid]) / BM + 1) / 2);
            if (tid < kMaxExperts) S.ptp[tid + 1] = v;
            if (tid == 0) S.ptp[0] = 0;
            __syncthreads();
            for (int off = 1; off < kMaxExperts; off <<= 1) {  // inclusive scan of S.ptp[1..256]
                int add = 0;
                if (tid >= off && tid < kMaxExperts) add = S.ptp[tid + 1 - off];
                __syncthreads();
                if (tid < kMaxExperts) S.ptp[tid + 1] += add;
                __syncthreads();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (C::PAIR && !C::FP4) cluster_sync();  // as above
    tc_fence_after();
    const uint32_t tmem_base = *S.tmem_slot;
    volatile int* abort_flag = S.abort_flag;

    // the padded layout: offsets start at 0, never decrease, every segment is a whole number
    // of 128-row tiles and the last ends within the row capacity; anything else is reported
    // and the launch does no work (the same decision in every CTA)
    bool bad_offs = false;
    if (P.row_offsets && tid < P.E) {
        const int64_t lo = S.offs[tid], hi = S.offs[tid + 1];
        bad_offs = hi < lo || (hi - lo) % BM != 0 || (tid == 0 && lo != 0);
    }
    bool layout_ok = !__syncthreads_or(bad_offs);
    if (P.row_offsets && S.offs[P.E] > P.rows) layout_ok = false;
    if (!layout_ok && tid == 0) record_error(P.status, MOE_ERR_BAD_INDEX, 20);
    const int64_t ntiles = layout_ok ? total_tiles<C>(P, S) : 0;

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------------------ TMA producer
        if constexpr (!C::FP4) {
            tma_prefetch_desc(&ma0);
            tma_prefetch_desc(&mb0);
            if (C::TWO_K || C::WGRAD) tma_prefetch_desc(&ma1);
            if (C::TWO_K || C::DUAL) tma_prefetch_desc(&mb1);
        }
        int stage = 0, expert = 0;
        uint32_t phase = 0;
        for (int64_t tile = first_tile; tile < ntiles; tile += tile_step) {
            const TileInfo ti = next_tile<C>(tile, expert, P, S, rank);
            bool ok = true;
            for (int kb = 0; kb < ti.k_iters; ++kb) {
                if (!mbar_wait_bounded(smem_u32(&S.empty[stage]), phase ^ 1u, abort_flag, P.status,
                                       P.wait_limit_ns, 30)) {
                    ok = false;
                    break;
                }
                const uint32_t full = smem_u32(&S.full[stage]);
                uint32_t bar = full;
                if constexpr (C::PAIR) {
                    bar = mapa_shared(full, 0);  // both CTAs' copies complete on the leader's
                    if (leader) mbar_arrive_expect_tx(full, 2 * (C::STAGE_BYTES - C::SF_BYTES));
                } else {
                    mbar_arrive_expect_tx(full, C::STAGE_BYTES - C::SF_BYTES);
                }
                const uint32_t a_dst = smem_u32(S.a + (size_t)stage * C::A_BYTES);
                const uint32_t b_dst = smem_u32(S.b + (size_t)stage * C::B_BYTES);
                if constexpr (C::FP4) {
                    uint32_t sf_bar = smem_u32(&S.sffull[stage]);
                    if (leader) mbar_arrive_expect_tx(sf_bar, (C::PAIR ? 2 : 1) * C::SF_BYTES);
                    if constexpr (C::PAIR) sf_bar = mapa_shared(sf_bar, 0);
                    issue_loads_fp4<C>(ti, kb, a_dst, b_dst,
                                       smem_u32(S.sf + (size_t)stage * C::SF_BYTES), bar, sf_bar, P,
                                       &ma0, &mb0, &mb1, msa, msb0, msb1, rank);
                } else
                    issue_loads<C>(ti, kb, a_dst, b_dst, bar, P, &ma0, &ma1, &mb0, &mb1, rank);
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
        }
    } else if (warp == 1 && lane == 0 && leader) {
        // ------------------------------------------------------------ MMA issuer
        int stage = 0;
        uint32_t phase = 0;
        int local = 0;
        uint32_t blocks = 0;  // K blocks so far (E2M1: buffer and phase of the scales)
        const uint32_t a_lo0 = desc_lo_sw128(smem_u32(S.a)), b_lo0 = desc_lo_sw128(smem_u32(S.b));
        for (int64_t tile = first_tile; tile < ntiles; tile += tile_step, ++local) {
            int k_iters, n0 = 0;
            if constexpr (C::FP4) {
                k_iters = (P.K0 + C::KB - 1) / C::KB;
                if (C::BN % 128) n0 = (int)((uint32_t)tile % (uint32_t)col_tiles<C>(P)) * C::BN;
            } else {
                k_iters = decode<C>(tile, P, S, rank).k_iters;
            }
            const int buf = local & 1;
            const uint32_t use = (local >> 1) & 1;
            if (!mbar_wait_bounded(smem_u32(&S.tempty[buf]), use ^ 1u, abort_flag, P.status,
                                   P.wait_limit_ns, 31))
                break;
            if constexpr (C::OV > 0)  // the columns shared with the previous tile's accumulator
                if (local > 0 && !mbar_wait_bounded(smem_u32(S.tshared), (local - 1) & 1, abort_flag,
                                                    P.status, P.wait_limit_ns, 35))
                    break;
            tc_fence_after();
            const uint32_t d_tmem = tmem_base + (buf ? C::ACC1 : C::ACC0);
            bool ok = true;
            for (int kb = 0; kb < k_iters; ++kb) {
                if (!mbar_wait_bounded(smem_u32(&S.full[stage]), phase, abort_flag, P.status,
                                       P.wait_limit_ns, 32)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if constexpr (C::FP4) {
                    // One thread issues everything, and what it takes to issue a block (two waits,
                    // four steps, a commit) is near what the block's products take: descriptors
                    // are one addition each, and a whole block has no branches.
                    const uint32_t sf = tmem_base + (blocks & 1) * C::SFC;
                    // 192 columns may begin in the middle of a scale tile: two words (of 32 rows) on
                    const uint32_t sfb = sf + C::SFK * 4 + (C::BN % 128 ? n0 % 128 / 32 : 0);
                    const uint32_t a_lo = a_lo0 + stage * (C::A_BYTES / 16);
                    const uint32_t b_lo = b_lo0 + stage * (C::B_BYTES / 16);
                    if (!mbar_wait_bounded(smem_u32(&S.sfready[blocks & 1]), (blocks >> 1) & 1,
                                           abort_flag, P.status, P.wait_limit_ns, 36)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    issue_step_fp4<C, 0>(d_tmem, sf, sfb, a_lo, b_lo, kb > 0);
                    issue_step_fp4<C, 1>(d_tmem, sf, sfb, a_lo, b_lo, 1);
                    if (P.K0 - kb * C::KB > 128) {  // K is a multiple of 128
                        issue_step_fp4<C, 2>(d_tmem, sf, sfb, a_lo, b_lo, 1);
                        issue_step_fp4<C, 3>(d_tmem, sf, sfb, a_lo, b_lo, 1);
                    }
                    ++blocks;
                } else {
                    const uint32_t a_s = smem_u32(S.a + (size_t)stage * C::A_BYTES);
                    const uint32_t b_s = smem_u32(S.b + (size_t)stage * C::B_BYTES);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {  // 4 instructions of 32 bytes of K
                        const uint64_t adesc = C::A_MN ? sdesc_sw128(a_s + kk * 2048, 8192, 1024)
                                                       : sdesc_sw128(a_s + kk * 32, 16, 1024);
                        const uint64_t bdesc = C::B_MN ? sdesc_sw128(b_s + kk * 2048, 8192, 1024)
                                                       : sdesc_sw128(b_s + kk * 32, 16, 1024);
                        const uint32_t acc = (kb > 0 || kk > 0) ? 1u : 0u;
                        if constexpr (C::PAIR && C::FP8) umma_fp8_pair(d_tmem, adesc, bdesc, C::IDESC, acc);
                        else if constexpr (C::PAIR) umma_bf16_pair(d_tmem, adesc, bdesc, C::IDESC, acc);
                        else if constexpr (C::FP8) umma_fp8(d_tmem, adesc, bdesc, C::IDESC, acc);
                        else umma_bf16(d_tmem, adesc, bdesc, C::IDESC, acc);
                    }
                }
                if constexpr (C::PAIR) umma_commit_pair(smem_u32(&S.empty[stage]), 0x3);
                else umma_commit(smem_u32(&S.empty[stage]));
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
            if constexpr (C::PAIR) umma_commit_pair(smem_u32(&S.tfull[buf]), 0x3);
            else umma_commit(smem_u32(&S.tfull[buf]));
        }
    } else if (C::FP4 && (warp == 2 || warp == 3) && lane == 0 && leader) {
        // ------------------------------------------------------------ scales to tensor memory
        if constexpr (C::FP4) {
            static_assert(C::STAGES >= 3, "a stage's phase while its scales' buffer is awaited");
            int stage = 0, old_stage = 0;
            uint32_t phase = 0, old_phase = 0, blocks = 0;
            const uint32_t sf_lo0 = desc_lo(smem_u32(S.sf));
            bool ok = true;
            const int k_iters = (P.K0 + C::KB - 1) / C::KB;
            for (int64_t tile = first_tile; ok && tile < ntiles; tile += tile_step) {
                for (int kb = 0; kb < k_iters; ++kb, ++blocks) {
                    // the products that read this buffer's last scales are those of two blocks
                    // ago, whose end frees their stage: no barrier of its own. (That stage's next
                    // use ends only after this thread has come past it, so the phase is unique.)
                    ok = mbar_wait_bounded(smem_u32(&S.sffull[stage]), phase, abort_flag, P.status,
                                           P.wait_limit_ns, 37) &&
                         (blocks < 2 ||
                          mbar_wait_bounded(smem_u32(&S.empty[old_stage]), old_phase, abort_flag,
                                            P.status, P.wait_limit_ns, 38));
                    if (!ok) break;
                    tc_fence_after();
                    const int left = (P.K0 - kb * C::KB) / 64;
                    issue_scales_fp4<C>(tmem_base + (blocks & 1) * C::SFC,
                                        sf_lo0 + stage * (C::SF_BYTES / 16), left < 4 ? left : 4,
                                        warp - 2);
                    if constexpr (C::PAIR) umma_commit_pair(smem_u32(&S.sfready[blocks & 1]), 0x1);
                    else umma_commit(smem_u32(&S.sfready[blocks & 1]));
                    if (blocks >= 2 && ++old_stage == C::STAGES) {
                        old_stage = 0;
                        old_phase ^= 1u;
                    }
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ epilogue
        const int q = warp % 4;  // TMEM lanes 32q .. 32q+31 (a warp's rank in its warpgroup)
        const int row_in_tile = 32 * q + lane;
        constexpr int kCols = C::BN / (C::EW / 4);  // columns per epilogue warp
        static_assert(kCols % 32 == 0, "epilogue column split");
        const int c_lo = ((warp - 4) / 4) * kCols;
        const int slot = warp - 4;
        uint32_t n_au = 0;  // staged a/u chunks consumed by this warp
        int local = 0, expert = 0;
        float* cs = S.cs + slot * C::CS_FLOATS;
        TileInfo following{};  // NV: the next tile
        float g_row = 1.0f, g_next = 1.0f;
        if constexpr (C::NV) {
            if (first_tile < ntiles) {
                following = next_tile<C>(first_tile, expert, P, S, rank);
                g_next = start_powers<C>(cs, P, following, row_in_tile, c_lo, lane);
            }
        }
        for (int64_t tile = first_tile; tile < ntiles; tile += tile_step, ++local) {
            const TileInfo ti = C::NV ? following : next_tile<C>(tile, expert, P, S, rank);
            const bool more = C::NV && tile + tile_step < ntiles;
            if (more) following = next_tile<C>(tile + tile_step, expert, P, S, rank);
            g_row = g_next;
            auto next_powers = [&] {
                if constexpr (C::NV)
                    if (more) g_next = start_powers<C>(cs, P, following, row_in_tile, c_lo, lane);
            };
            const int buf = local & 1;
            const uint32_t ph = (local >> 1) & 1;
            Readers rd{};
            if constexpr (C::FP4) {  // buffer 0 shares its last columns, buffer 1 its first
                const int group = (warp - 4) / 4;
                rd.shared = buf == 0 ? group >= C::EW / 4 - C::OV_GROUPS : group < C::OV_GROUPS;
                rd.shared_bar = smem_u32(S.tshared);
                rd.whole_bar = smem_u32(&S.tempty[buf]);
                if constexpr (C::PAIR) {
                    rd.shared_bar = mapa_shared(rd.shared_bar, 0);
                    rd.whole_bar = mapa_shared(rd.whole_bar, 0);
                }
            }
            if constexpr (C::AU && C::FP4) {
                if (lane == 0)
                    au_issue_fp4<C>(S, &ma1, &mb1, slot, ti.m0 + 32 * q, ti.n0 + c_lo);
            } else if constexpr (C::AU) {  // this tile's first a/u chunks while the MMA runs
                if (lane == 0)
                    for (int i = 0; i < kAuBufs && i < kCols / kAuCols; ++i)
                        au_issue<C>(S, &ma1, &mb1, slot, n_au + i, ti.m0 + 32 * q,
                                    ti.n0 + c_lo + i * kAuCols);
            }
            bool apart = false;  // NV: powers that are not multiplied with one another
            if constexpr (C::NV) {
                cp_async_wait_all();
                __syncwarp();
                if (ti.m0 < ti.row_end && (C::BN % 128 == 0 || ti.n0 + c_lo < P.N))  // (else it has none)
                    apart = !powers_multiply<C>(cs, g_row, lane);
            }
            bool ok = mbar_wait_bounded(smem_u32(&S.tfull[buf]), ph, abort_flag, P.status,
                                        P.wait_limit_ns, 33);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const uint32_t t_acc =
                tmem_base + (buf ? C::ACC1 : C::ACC0) + ((uint32_t)(32 * q) << 16);
            if constexpr (C::NV)
                if (apart) {
                    scale_in_place<C>(t_acc + c_lo, g_row, cs, lane);
                    g_row = 1.0f;
                }
            if constexpr (C::AU && C::FP4) {
                if (!swiglu_bwd_fp4<C>(S, ti, t_acc, q, lane, slot, c_lo, P, &mo0, &mo1,
                                       (uint32_t)local, abort_flag, g_row, cs, next_powers))
                    break;
            } else if constexpr (C::AU) {
                if (!swiglu_bwd_staged<C>(S, ti, t_acc, q, lane, slot, c_lo, kCols, P, &ma1, &mb1,
                                          &mo0, &mo1, n_au, abort_flag))
                    break;
            } else if constexpr (C::FP4) {
                epilogue_fp4<C>(S, ti, t_acc, lane, slot, c_lo, ti.m0 + 32 * q, P, &mo0, &mo1, &mo2,
                                buf == 0, rd, g_row, cs, next_powers);
                continue;
            } else if constexpr (C::TS) {
                epilogue_tma_store<C>(S, ti, t_acc, q, lane, slot, c_lo, kCols, P, &mo0, &mo1, &mo2,
                                      n_au);
            } else {
                epilogue_wgrad<C>(ti, t_acc, row_in_tile, P, c_lo, c_lo + kCols);
            }
            if constexpr (C::FP4) {
                arrive_read<C>(rd.whole_bar, lane);
                continue;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (C::PAIR) mbar_arrive_cluster(mapa_shared(smem_u32(&S.tempty[buf]), 0));
                else mbar_arrive(smem_u32(&S.tempty[buf]));
            }
        }
        if constexpr (C::NV) cp_async_wait_all();  // (a wait that ran out leaves one under way)
        if constexpr (C::TS) {
            if (lane == 0) bulk_wait<0>();  // this warp's stores are complete
        }
    }
    __syncwarp();
    __syncthreads();
    if constexpr (C::PAIR) cluster_sync();  // no CTA leaves while its peer may still signal it
    if (*abort_flag) {  // let copies still in flight land before the CTA exits
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000ull) {
        }
    }
    if (warp == 2) {
        tc_fence_after();
        if constexpr (C::PAIR) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
        else tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap ma0,
                        const __grid_constant__ CUtensorMap ma1,
                        const __grid_constant__ CUtensorMap mb0,
                        const __grid_constant__ CUtensorMap mb1,
                        const __grid_constant__ CUtensorMap mo0,
                        const __grid_constant__ CUtensorMap mo1,
                        const __grid_constant__ CUtensorMap mo2, const Params P) {
    grouped_gemm_body<C>(ma0, ma1, mb0, mb1, mo0, mo1, mo2, nullptr, nullptr, nullptr, P);
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    grouped_gemm_fp4_kernel(const __grid_constant__ CUtensorMap ma0,
                            const __grid_constant__ CUtensorMap ma1,
                            const __grid_constant__ CUtensorMap mb0,
                            const __grid_constant__ CUtensorMap mb1,
                            const __grid_constant__ CUtensorMap mo0,
                            const __grid_constant__ CUtensorMap mo1,
                            const __grid_constant__ CUtensorMap mo2,
                            const __grid_constant__ CUtensorMap msa,
                            const __grid_constant__ CUtensorMap msb0,
                            const __grid_constant__ CUtensorMap msb1, const Params P) {
    grouped_gemm_body<C>(ma0, ma1, mb0, mb1, mo0, mo1, mo2, &msa, &msb0, &msb1, P);
}

// ---------------------------------------------------------------------- host side

PFN_cuTensorMapEncodeTiled_v12000 get_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// 2-D map over a row-major [outer, inner] matrix of bf16 (or of bytes, for E4M3 codes),
// 128-byte swizzled boxes.
bool make_map(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer,
              uint32_t box_inner, uint32_t box_outer, bool bytes = false,
              CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B) {
    auto enc = get_encoder();
    if (!enc || !base) return false;
    cuuint64_t dims[2] = {inner, outer};
    cuuint64_t strides[1] = {inner * (bytes ? 1 : 2)};
    cuuint32_t box[2] = {box_inner, box_outer};
    cuuint32_t es[2] = {1, 1};
    return enc(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
               const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor maps for the TMA-store epilogue: boxes of `cols` (16, 32 or 64) x 32 rows over [rows, ld]
// bf16, swizzled as the epilogue lays them out (32-, 64- or 128-byte rows).
bool out_maps(CUtensorMap (&mo)[3], const void* o0, const void* o1, const void* o2, uint64_t ld,
              uint64_t rows, int cols = kOutCols) {
    const void* o[3] = {o0, o1, o2};
    const CUtensorMapSwizzle swz = cols == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                   : cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                : CU_TENSOR_MAP_SWIZZLE_32B;
    for (int i = 0; i < 3; ++i)  // (what is not given is not written)
        if (!o[i] && i) mo[i] = mo[0];
        else if (!make_map(&mo[i], o[i], ld, rows, (uint32_t)cols, 32, false, swz)) return false;
    return true;
}

// `mo` (TMA-store configurations only): the output maps from out_maps. `sf` (E2M1 only): the maps
// of A's, the first and the second B operand's scale tiles.
template <class C>
int launch(const CUtensorMap& a0, const CUtensorMap& a1, const CUtensorMap& b0,
           const CUtensorMap& b1, const Params& P, int64_t max_tiles, cudaStream_t st,
           const CUtensorMap* mo = nullptr, const CUtensorMap* sf = nullptr) {
    static_assert(C::SMEM_BYTES <= 227 * 1024, "shared memory");
    if ((C::TS && !mo) || (C::FP4 && !sf)) return MOE_ERR_LAUNCH;
    const CUtensorMap& o0 = mo ? mo[0] : a0;
    const CUtensorMap& o1 = mo ? mo[1] : a0;
    const CUtensorMap& o2 = mo ? mo[2] : a0;
    auto kern = [] {
        if constexpr (C::FP4) return grouped_gemm_fp4_kernel<C>;
        else return grouped_gemm_kernel<C>;
    }();
    // What the runtime says of a kernel on a device does not change: asked once for each. (E2M1; a call
    // for one token is mostly the host's work.)
    static std::atomic<int> resident[C::FP4 ? kMaxDevices : 1];
    int dev = 0;
    if (C::FP4 && (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices))
        return MOE_ERR_LAUNCH;
    int clusters = C::FP4 ? resident[dev].load(std::memory_order_acquire) : 0;
    if (clusters == 0 && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              (int)C::SMEM_BYTES) != cudaSuccess)
        return MOE_ERR_LAUNCH;
    if constexpr (C::PAIR) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.blockDim = dim3(C::THREADS);
        cfg.dynamicSmemBytes = C::SMEM_BYTES;
        cfg.stream = st;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        cfg.gridDim = dim3(2 * (unsigned)(sm_count() / 2));
        if (clusters == 0) {  // pairs that fit on the GPU at once (one CTA per SM)
            if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) != cudaSuccess || clusters < 1)
                clusters = sm_count() / 2;
            if (C::FP4) resident[dev].store(clusters, std::memory_order_release);
        }
        int64_t pairs = clusters;
        if (max_tiles < pairs) pairs = max_tiles;
        if (pairs < 1) pairs = 1;
        cfg.gridDim = dim3(2 * (unsigned)pairs);
        cudaError_t rc;
        if constexpr (C::FP4) {
            attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[1].val.programmaticStreamSerializationAllowed = 1;
            cfg.numAttrs = 2;
        }
        if constexpr (C::FP4)
            rc = cudaLaunchKernelEx(&cfg, kern, a0, a1, b0, b1, o0, o1, o2, sf[0], sf[1], sf[2], P);
        else
            rc = cudaLaunchKernelEx(&cfg, kern, a0, a1, b0, b1, o0, o1, o2, P);
        if (rc != cudaSuccess) return MOE_ERR_LAUNCH;
        return launch_status();
    } else {
        int64_t grid = sm_count();
        if (max_tiles < grid) grid = max_tiles;
        if (grid < 1) grid = 1;
        if constexpr (C::FP4) {
            if (clusters == 0) resident[dev].store(1, std::memory_order_release);  // the attribute is set
            return launch_dependent(kern, dim3((unsigned)grid), dim3(C::THREADS), C::SMEM_BYTES, st, a0,
                                    a1, b0, b1, o0, o1, o2, sf[0], sf[1], sf[2], P);
        } else {
            kern<<<(unsigned)grid, C::THREADS, C::SMEM_BYTES, st>>>(a0, a1, b0, b1, o0, o1, o2, P);
            return launch_status();
        }
    }
}

Params base_params(const int64_t* row_offsets, int64_t rows, int E) {
    Params P{};
    P.row_offsets = row_offsets;
    P.rows = rows;
    P.E = E;
    P.status = device_status_word();
    P.wait_limit_ns = wait_limit_ns();
    return P;
}

int64_t token_tiles_max(int64_t rows, int N, int BN) { return cdiv(rows, BM) * cdiv(N, BN); }

bool gemm_shape_ok(int d, int f) { return d % 128 == 0 && f % 128 == 0 && d > 0 && f > 0; }

}  // namespace
}  // namespace moe
