// Quantisation to microscaled 4-bit floating point and back, and the dispatch of quantised rows
// (the formats: fp4.cuh). All four are bound by memory. They are launched behind one another
// (launch_dependent), as are the GEMMs that read what they make: a token's chain of short kernels
// is set up while the one before ends.
#include <cuda_fp4.h>
#include <cuda_runtime.h>

#include "fp4.cuh"
#include "sizes.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Rows. A thread takes 16 consecutive elements (32 bytes) at a time and keeps up to NIT such
// pieces in registers, so that a row is read once although its largest value (NV) is needed
// first. TPR threads share a row. Blocks of 16 lie in one thread, blocks of 32 in two; the four
// scales of a tile's row are put together by shuffles and stored as one word.
// 65,535 x 4096 (MX): 107 us, 0.94 of the copy rate over 0.68 GB.
template <bool NV, int TPR, int NIT>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(
    const __nv_bfloat16* __restrict__ X, const __nv_bfloat16* __restrict__ X1,
    const int64_t* __restrict__ limit, int64_t rows, int cols, uint8_t* __restrict__ Q,
    uint8_t* __restrict__ S, float* __restrict__ G) {
    grid_launch_dependents();
    grid_dependency_wait();
    constexpr int ROWS = kThreads / TPR;  // rows a CTA takes at a time
    static_assert(TPR <= 32 || TPR == kThreads, "a row in one warp or in the whole CTA");
    __shared__ uint32_t part[NV && TPR > 32 ? kThreads / 32 : 1];
    const int lane = threadIdx.x % 32;
    const int t = threadIdx.x % TPR;
    const int np0 = cols / 16;                 // pieces of X's row
    const int np = X1 ? 2 * np0 : np0;
    const int64_t ktiles = np * 16 / Fp4<NV>::TILE_K;
    int64_t n = rows;
    if (limit) n = min(n, *limit);
    for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < n; r0 += (int64_t)gridDim.x * ROWS) {
        const int64_t r = r0 + threadIdx.x / TPR;
        const bool in_row = r < n;
        uint4 v[NIT][2];
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            const int p = t + i * TPR;
            v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
            if (in_row && p < np) {
                const __nv_bfloat16* src = p < np0 ? X + r * cols + 16 * p
                                                   : X1 + r * cols + 16 * (p - np0);
                v[i][0] = reinterpret_cast<const uint4*>(src)[0];
                v[i][1] = reinterpret_cast<const uint4*>(src)[1];
            }
        }
        uint32_t am[NIT];
#pragma unroll
        for (int i = 0; i < NIT; ++i) am[i] = halves_max(absmax8(absmax8(0u, v[i][0]), v[i][1]));
        uint32_t top = 0;
        if constexpr (NV) {
#pragma unroll
            for (int i = 0; i < NIT; ++i) top = max(top, am[i]);
            if constexpr (TPR >= 32) {
                top = __reduce_max_sync(0xffffffffu, top);
            } else {
#pragma unroll
                for (int o = TPR / 2; o > 0; o >>= 1)
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            }
            if constexpr (TPR > 32) {
                if (lane == 0) part[threadIdx.x / 32] = top;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < kThreads / 32; ++w) top = max(top, part[w]);
                __syncthreads();
            }
        }
        const NvRow row(top);
        if (NV && in_row && t == 0) G[r] = row.g;
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            const int p = t + i * TPR;
            if (i * TPR >= np) break;  // the same for the whole CTA
            uint2 code;
            uint32_t word;
            if constexpr (NV) {
                const NvScale sc(am[i], row);
                code = make_uint2(sc.codes(v[i][0]), sc.codes(v[i][1]));
                word = sc.byte << (8 * (lane & 3));
                word |= __shfl_xor_sync(0xffffffffu, word, 1);
                word |= __shfl_xor_sync(0xffffffffu, word, 2);
            } else {
                const MxScale sc(max(am[i], __shfl_xor_sync(0xffffffffu, am[i], 1)));
                code = make_uint2(sc.codes(v[i][0]), sc.codes(v[i][1]));
                word = sc.byte << (8 * ((lane >> 1) & 3));
                word |= __shfl_xor_sync(0xffffffffu, word, 2);
                word |= __shfl_xor_sync(0xffffffffu, word, 4);
            }
            if (in_row && p < np) {  // np is a multiple of 8: whole tiles of scales
                reinterpret_cast<uint2*>(Q + r * (np * 8))[p] = code;
                constexpr int PT = Fp4<NV>::TILE_K / 16;  // pieces of a tile
                if (lane % PT == 0)
                    *reinterpret_cast<uint32_t*>(S + fp4_scale_word(r, p / PT, ktiles)) = word;
            }
        }
    }
}

// The numbers that codes stand for: E2M1 * scale (* g), one rounding to bf16, which is exact (the
// product has at most 6 significant bits) unless it leaves bf16's range. A thread makes 8 numbers,
// 16 bytes, so that a warp's store is one run of 512 (with 32 bytes a thread the two stores of a
// sector's halves made 65,535 x 4096 134 us; now 114, 0.88 of the copy rate, the issue slots 80% in use).
// `Index` counts pieces of 8; 32 bits where they do.
template <bool NV, class Index>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(
    const uint8_t* __restrict__ Q, const uint8_t* __restrict__ S, const float* __restrict__ G,
    const int64_t* __restrict__ limit, int64_t rows, int cols, __nv_bfloat16* __restrict__ out) {
    grid_launch_dependents();
    grid_dependency_wait();
    const Index np = cols / 8;
    const int64_t ktiles = cols / Fp4<NV>::TILE_K;
    constexpr int PB = Fp4<NV>::BLOCK / 8;  // pieces of a block
    constexpr int U = 4;                    // pieces a thread has in flight
    int64_t n = rows;
    if (limit) n = min(n, *limit);
    const int64_t total = n * np;
    for (int64_t i0 = (int64_t)blockIdx.x * kThreads * U + threadIdx.x; i0 < total;
         i0 += (int64_t)gridDim.x * kThreads * U) {
        uint32_t code[U], byte[U];
        float g[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * kThreads;
            code[u] = byte[u] = 0;
            g[u] = 1.0f;
            if (i >= total) continue;
            const Index r = (Index)i / np, p = (Index)i - r * np;
            code[u] = reinterpret_cast<const uint32_t*>(Q)[i];
            byte[u] = S[fp4_scale_word(r, p / (4 * PB), ktiles) + p / PB % 4];
            if (NV) g[u] = G[r];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * kThreads;
            if (i >= total) break;
            float s;
            if constexpr (NV)
                s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte[u], __NV_E4M3))) * g[u];
            else
                s = byte[u] == 255 ? __uint_as_float(0x7fffffffu)
                                   : byte[u] ? __uint_as_float(byte[u] << 23) : __uint_as_float(1u << 22);
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t b = (code[u] >> (8 * j)) & 0xffu;
                const __half2 h(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)b, __NV_E2M1));
                const float2 f = __half22float2(h);
                w[j] = pack_bf16x2(f.x * s, f.y * s);
            }
            reinterpret_cast<uint4*>(out)[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ------------------------------------------------ columnwise scales, transposed codes
// X is E matrices of K x N bf16, or, with X1, the K = 2 K0 stack of X0 over X1. Column n's codes
// are written as row e N + n of the operand, K-major, its blocks along K.

// A CTA takes a strip of NC columns and KT rows through shared memory: all K rows in NV, whose columns'
// largest values are needed first, so that X is read once; 256 rows in MX. A thread then makes the
// codes of 32 K elements (a piece) of two neighbouring columns, whose values lie in one word a row;
// they go back through shared memory to leave as whole lines. NV operands whose strips are too long
// for that (K over kStripMaxK) get the columns' largest values from a pass of its own.
// 128 stacks of 1536 x 2048 (MX): 186 us, 0.80 of the copy rate over 1.0 GB. 64 matrices of 1024 x 256
// (NV): 23 us over 43 MB; a CTA loads, then computes, and few CTAs are at a time in either.
constexpr int kStripRowsMx = 256;
constexpr int kStripRowsNv = 512;  // after that pass
constexpr int kStripMaxK = 3328;

// A strip in shared memory, in words of two columns: rows padded by one word and pieces of 32 rows by
// NC / 2, so that the rows a warp's lanes read at once, 32 apart, lie in different banks.
template <int NC>
struct Strip {
    static constexpr int W = NC / 2;
    static constexpr int PIECE = 32 * (W + 1) + W;
    __device__ __forceinline__ static int word(int r) { return r / 32 * PIECE + r % 32 * (W + 1); }
    static size_t bytes(int rows) { return (size_t)rows / 32 * PIECE * 4; }
};

template <bool NV, int NC>
__global__ void __launch_bounds__(kThreads, 4) quantize_cols_kernel(
    const __nv_bfloat16* __restrict__ X0, const __nv_bfloat16* __restrict__ X1, int K0, int N, int KT,
    uint8_t* __restrict__ Qt, uint8_t* __restrict__ S, float* __restrict__ G, bool have_g) {
    grid_launch_dependents();
    grid_dependency_wait();
    extern __shared__ __align__(16) uint8_t strip_smem[];
    using L = Strip<NC>;
    constexpr int WORD_K = Fp4<NV>::TILE_K;
    uint32_t* tile = reinterpret_cast<uint32_t*>(strip_smem);
    __shared__ uint32_t top[NC];
    const int K = X1 ? 2 * K0 : K0;
    const int e = blockIdx.z, n0 = blockIdx.x * NC, k0 = blockIdx.y * KT;
    const int kn = min(KT, K - k0);  // a multiple of 128
    if (NV && threadIdx.x < NC) top[threadIdx.x] = 0;
    if (NV) __syncthreads();
    // in: 16 bytes (8 columns) a thread and row
    constexpr int V = NC / 8;
    const int c8 = threadIdx.x % V;
    uint4 m = make_uint4(0, 0, 0, 0);
    constexpr int U = 8;  // rows a thread has in flight
    for (int r0 = threadIdx.x / V; r0 < kn; r0 += U * (kThreads / V)) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * (kThreads / V), k = k0 + r;
            v[u] = make_uint4(0, 0, 0, 0);
            if (r < kn)
                v[u] = *reinterpret_cast<const uint4*>(
                    (k < K0 ? X0 + ((int64_t)e * K0 + k) * N : X1 + ((int64_t)e * K0 + (k - K0)) * N) + n0 + 8 * c8);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * (kThreads / V);
            if (r >= kn) break;
            uint32_t* dst = tile + L::word(r) + 4 * c8;
            dst[0] = v[u].x;
            dst[1] = v[u].y;
            dst[2] = v[u].z;
            dst[3] = v[u].w;
            if (NV)
                m = make_uint4(absmax2(m.x, v[u].x), absmax2(m.y, v[u].y), absmax2(m.z, v[u].z),
                               absmax2(m.w, v[u].w));
        }
    }
    if (NV && !have_g) {  // a warp's rows first, or its lanes would queue at the same few words
        uint32_t w[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int o = 16; o >= V; o >>= 1) w[q] = __vmaxu2(w[q], __shfl_xor_sync(0xffffffffu, w[q], o));
            if (threadIdx.x % 32 < V) {
                atomicMax(&top[8 * c8 + 2 * q], w[q] & 0xffffu);
                atomicMax(&top[8 * c8 + 2 * q + 1], w[q] >> 16);
            }
        }
    }
    __syncthreads();
    // codes: columns 2 p and 2 p + 1, rows from 32 q on; QN pieces a round, whose codes then take the
    // place of the rows they were made of
    constexpr int QN = kThreads / L::W;
    const int p = threadIdx.x % L::W;
    const int64_t r = (int64_t)e * N + n0 + 2 * p;
    NvRow row0(0), row1(0);
    if (NV) {
        if (have_g) {
            row0.g = G[r], row1.g = G[r + 1];
            row0.inv = 1.0f / row0.g, row1.inv = 1.0f / row1.g;  // of powers of two: exact
        } else {
            row0 = NvRow(top[2 * p]), row1 = NvRow(top[2 * p + 1]);
            if (threadIdx.x < L::W) G[r] = row0.g, G[r + 1] = row1.g;
        }
    }
    for (int q0 = 0; q0 < kn / 32; q0 += QN) {
        const int np = min(QN, kn / 32 - q0);  // pieces of this round
        const int q = threadIdx.x / L::W;
        uint32_t code[2][4] = {};
        if (q < np) {
            const uint32_t* src = tile + L::word(32 * (q0 + q)) + p;
            const int64_t kk = k0 + 32 * (q0 + q);
            uint8_t* s0 = S + fp4_scale_word(r, kk / WORD_K, K / WORD_K) + kk % WORD_K / Fp4<NV>::BLOCK;
            uint8_t* s1 = S + fp4_scale_word(r + 1, kk / WORD_K, K / WORD_K) + kk % WORD_K / Fp4<NV>::BLOCK;
            constexpr int B = Fp4<NV>::BLOCK;
            uint32_t bytes0 = 0, bytes1 = 0;
#pragma unroll
            for (int h = 0; h < 32 / B; ++h) {  // blocks of the piece
                uint32_t v[B], am = 0;
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    v[i] = src[(h * B + i) * (L::W + 1)];
                    am = absmax2(am, v[i]);
                }
                auto make = [&](const auto& sa, const auto& sb) {
                    bytes0 |= sa.byte << (8 * h);
                    bytes1 |= sb.byte << (8 * h);
#pragma unroll
                    for (int j = 0; j < B / 8; ++j) {
                        float a[8], b[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            a[i] = sa.quot(bf16_lo(v[8 * j + i]));
                            b[i] = sb.quot(bf16_hi(v[8 * j + i]));
                        }
                        code[0][h * (B / 8) + j] = sa.finish(fp4_codes8(a));
                        code[1][h * (B / 8) + j] = sb.finish(fp4_codes8(b));
                    }
                };
                if constexpr (NV) make(NvScale(am & 0xffffu, row0), NvScale(am >> 16, row1));
                else make(MxScale(am & 0xffffu), MxScale(am >> 16));
            }
            if constexpr (NV) {
                *reinterpret_cast<uint16_t*>(s0) = (uint16_t)bytes0;
                *reinterpret_cast<uint16_t*>(s1) = (uint16_t)bytes1;
            } else {
                *s0 = (uint8_t)bytes0;
                *s1 = (uint8_t)bytes1;
            }
        }
        __syncthreads();  // every row of this round has been read
        uint4* out = reinterpret_cast<uint4*>(tile + L::word(32 * q0));  // pieces are multiples of 16 bytes
        if (q < np) {
            out[2 * p * (np + 1) + q] = make_uint4(code[0][0], code[0][1], code[0][2], code[0][3]);
            out[(2 * p + 1) * (np + 1) + q] = make_uint4(code[1][0], code[1][1], code[1][2], code[1][3]);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < NC * np; i += kThreads) {
            const int col = i / np, piece = i - col * np;
            *reinterpret_cast<uint4*>(Qt + ((int64_t)e * N + n0 + col) * (K / 2) + (k0 + 32 * (q0 + piece)) / 2) =
                out[col * (np + 1) + piece];
        }
    }
}

// NV, long strips: largest magnitude of each column (as bits, which order as the magnitudes do; `top`
// starts at zero). A thread takes 8 columns of every sixteenth row.
constexpr int kTopRows = 256;

__global__ void __launch_bounds__(kThreads) column_top_kernel(const __nv_bfloat16* __restrict__ X0,
                                                              const __nv_bfloat16* __restrict__ X1,
                                                              int K0, int N, uint32_t* __restrict__ top) {
    const int e = blockIdx.y;
    const int K = X1 ? 2 * K0 : K0;
    const int c = blockIdx.x * 128 + threadIdx.x % 16 * 8;  // N is a multiple of 128
    const int r1 = min(K, (int)(blockIdx.z + 1) * kTopRows);
    uint4 m = make_uint4(0, 0, 0, 0);
#pragma unroll 8
    for (int r = blockIdx.z * kTopRows + threadIdx.x / 16; r < r1; r += kThreads / 16) {
        const __nv_bfloat16* src = r < K0 ? X0 + ((int64_t)e * K0 + r) * N
                                          : X1 + ((int64_t)e * K0 + (r - K0)) * N;
        const uint4 v = *reinterpret_cast<const uint4*>(src + c);
        m = make_uint4(absmax2(m.x, v.x), absmax2(m.y, v.y), absmax2(m.z, v.z), absmax2(m.w, v.w));
    }
    __shared__ uint32_t part[128];
    if (threadIdx.x < 128) part[threadIdx.x] = 0;
    __syncthreads();
    uint32_t w[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        w[q] = __vmaxu2(w[q], __shfl_xor_sync(0xffffffffu, w[q], 16));
        if (threadIdx.x % 32 < 16) {
            atomicMax(&part[threadIdx.x % 16 * 8 + 2 * q], w[q] & 0xffffu);
            atomicMax(&part[threadIdx.x % 16 * 8 + 2 * q + 1], w[q] >> 16);
        }
    }
    __syncthreads();
    if (threadIdx.x < 128) atomicMax(top + (int64_t)e * N + blockIdx.x * 128 + threadIdx.x, part[threadIdx.x]);
}

// Column maxima (bits) to the rows' powers of two, in place.
__global__ void column_g_kernel(float* __restrict__ G, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) G[i] = NvRow(__float_as_uint(G[i])).g;
}

// ---------------------------------------------------------- dispatch of quantised rows
// Codes and scales of a row depend on that row alone, so those of an expert-major row are its
// token's: a warp copies a token's codes and scale words to its k rows. 32,768 tokens of 2048 to 8 rows each
// (MX): 68 us for 0.34 GB (0.73 of the copy rate; the scale words, 4 bytes each, are what slows it:
// gathered into whole tiles by their destination they took longer).
// The CTAs behind those take the padding rows of each segment (the trailing rows with perm_token < 0;
// at most MOE_ROW_ALIGN - 1 per expert): zero codes, scales of zero bits and g = 1, as quantising a
// zero row gives.
constexpr int kPadSplit = 8;
constexpr int kSitePermuteFp4 = 21;

__global__ void __launch_bounds__(kThreads) permute_kernel(
    const uint8_t* __restrict__ xq, const uint8_t* __restrict__ sx, const float* __restrict__ gx,
    const int32_t* __restrict__ slot_to_row, const int32_t* __restrict__ perm_token,
    const int64_t* __restrict__ row_offsets, int64_t T, int64_t rows, int d, int k, int ktiles,
    int64_t token_ctas, uint8_t* __restrict__ Xq, uint8_t* __restrict__ sX, float* __restrict__ gX,
    int* __restrict__ status) {
    grid_launch_dependents();
    grid_dependency_wait();
    if (blockIdx.x >= token_ctas) {
        const int e = (int)(blockIdx.x - token_ctas) / kPadSplit, part = (int)(blockIdx.x - token_ctas) % kPadSplit;
        const int64_t hi = row_offsets[e + 1];
        int64_t lo = row_offsets[e];
        if (lo < 0 || hi < lo || hi > rows) {  // not a layout of these rows
            if (threadIdx.x == 0) record_error(status, MOE_ERR_BAD_INDEX, kSitePermuteFp4);
            return;
        }
        if (hi - lo > MOE_ROW_ALIGN - 1) lo = hi - (MOE_ROW_ALIGN - 1);
        for (int64_t r = lo + part * (kThreads / 32) + threadIdx.x / 32; r < hi;
             r += kPadSplit * (kThreads / 32)) {  // a warp a row
            if (perm_token[r] >= 0) continue;
            for (int c = threadIdx.x % 32; c < d / 32; c += 32)
                reinterpret_cast<uint4*>(Xq + r * (d / 2))[c] = make_uint4(0, 0, 0, 0);
            for (int c = threadIdx.x % 32; c < ktiles; c += 32)
                *reinterpret_cast<uint32_t*>(sX + fp4_scale_word(r, c, ktiles)) = 0;
            if (gX && threadIdx.x % 32 == 0) gX[r] = 1.0f;
        }
        return;
    }
    const int lane = threadIdx.x % 32;
    const int64_t t = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    if (t >= T) return;
    int32_t my_row = -1;
    if (lane < k) my_row = slot_to_row[t * k + lane];
    if (my_row >= rows) {
        record_error(status, MOE_ERR_BAD_INDEX, kSitePermuteFp4);
        my_row = -1;
    }
    if (gx && my_row >= 0) gX[my_row] = gx[t];
    const uint4* src = reinterpret_cast<const uint4*>(xq + t * (d / 2));
    const int nvec = d / 32;
    for (int c0 = 0; c0 < nvec; c0 += 32) {  // warp-uniform trip count
        const int c = c0 + lane;
        const bool in = c < nvec;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (in) v = src[c];
        for (int i = 0; i < k; ++i) {
            const int32_t row = __shfl_sync(0xffffffffu, my_row, i);
            if (in && row >= 0) reinterpret_cast<uint4*>(Xq + (int64_t)row * (d / 2))[c] = v;
        }
    }
    for (int c0 = 0; c0 < ktiles; c0 += 32) {
        const int c = c0 + lane;
        const bool in = c < ktiles;
        uint32_t w = 0;
        if (in) w = *reinterpret_cast<const uint32_t*>(sx + fp4_scale_word(t, c, ktiles));
        for (int i = 0; i < k; ++i) {
            const int32_t row = __shfl_sync(0xffffffffu, my_row, i);
            if (in && row >= 0)
                *reinterpret_cast<uint32_t*>(sX + fp4_scale_word(row, c, ktiles)) = w;
        }
    }
}

template <bool NV, int TPR, int NIT>
int launch_rows(const __nv_bfloat16* X, const __nv_bfloat16* X1, const int64_t* limit, int64_t rows,
                int cols, uint8_t* Q, uint8_t* S, float* g, cudaStream_t st) {
    int64_t blocks = cdiv(rows, kThreads / TPR);
    const int64_t cap = (int64_t)sm_count() * 16;
    if (blocks > cap) blocks = cap;
    return launch_dependent(quantize_rows_kernel<NV, TPR, NIT>, dim3((unsigned)blocks), dim3(kThreads), 0, st,
                            X, X1, limit, rows, cols, Q, S, g);
}

template <bool NV>
int rows_by_width(const __nv_bfloat16* X, const __nv_bfloat16* X1, const int64_t* limit, int64_t rows,
                  int cols, uint8_t* Q, uint8_t* S, float* g, cudaStream_t st) {
    const int width = X1 ? 2 * cols : cols;
    // A warp holds rows of up to 4096 elements; wider ones, and rows too few to fill the GPU with
    // a warp each, take a CTA of eight.
    if (width > 4096 || rows < 8 * (int64_t)sm_count()) {
        if (width <= 4096) return launch_rows<NV, 256, 1>(X, X1, limit, rows, cols, Q, S, g, st);
        if (width <= 8192) return launch_rows<NV, 256, 2>(X, X1, limit, rows, cols, Q, S, g, st);
        return launch_rows<NV, 256, 8>(X, X1, limit, rows, cols, Q, S, g, st);
    }
    // many narrow rows: few threads each, so that none idles
    if (width <= 512 && rows >= 256 * (int64_t)sm_count()) {
        if (width <= 256) return launch_rows<NV, 8, 2>(X, X1, limit, rows, cols, Q, S, g, st);
        return launch_rows<NV, 16, 2>(X, X1, limit, rows, cols, Q, S, g, st);
    }
    if (width <= 1024) return launch_rows<NV, 32, 2>(X, X1, limit, rows, cols, Q, S, g, st);
    if (width <= 2048) return launch_rows<NV, 32, 4>(X, X1, limit, rows, cols, Q, S, g, st);
    return launch_rows<NV, 32, 8>(X, X1, limit, rows, cols, Q, S, g, st);
}

template <bool NV, int NC>
int launch_cols(const __nv_bfloat16* X0, const __nv_bfloat16* X1, int E, int K0, int N, int K, int KT,
                uint8_t* Qt, uint8_t* S, float* g, bool have_g, cudaStream_t st) {
    const size_t smem = Strip<NC>::bytes(KT);
    auto kern = quantize_cols_kernel<NV, NC>;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return MOE_ERR_LAUNCH;
    return launch_dependent(kern, dim3((unsigned)(N / NC), (unsigned)cdiv(K, KT), (unsigned)E), dim3(kThreads),
                            smem, st, X0, X1, K0, N, KT, Qt, S, g, have_g);
}

template <bool NV>
int launch_dequantize(const uint8_t* Q, const uint8_t* S, const float* g, const int64_t* limit,
                       int64_t rows, int cols, __nv_bfloat16* out, cudaStream_t st) {
    const int64_t pieces = rows * (cols / 8);
    int64_t blocks = cdiv(pieces, 4 * kThreads);
    const int64_t cap = (int64_t)sm_count() * 32;
    if (blocks > cap) blocks = cap;
    auto kern = pieces < (int64_t(1) << 32) ? dequantize_kernel<NV, uint32_t> : dequantize_kernel<NV, int64_t>;
    return launch_dependent(kern, dim3((unsigned)blocks), dim3(kThreads), 0, st, Q, S, g, limit, rows, cols, out);
}

bool fmt_ok(int fmt) { return fmt == MOE_FP4_MX || fmt == MOE_FP4_NV; }
// NV has a power of two for each row, MX has none.
bool g_ok(int fmt, const float* g) { return (fmt == MOE_FP4_NV) == (g != nullptr); }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

int launch_quantize_rows_fp4(const __nv_bfloat16* X, const __nv_bfloat16* X1, const int64_t* limit,
                             int64_t rows, int cols, int fmt, uint8_t* Q, uint8_t* S, float* g,
                             cudaStream_t st) {
    return fmt == MOE_FP4_NV ? rows_by_width<true>(X, X1, limit, rows, cols, Q, S, g, st)
                             : rows_by_width<false>(X, X1, limit, rows, cols, Q, S, g, st);
}

}  // namespace moe

using namespace moe;

extern "C" int64_t moe_fp4_scale_bytes(int64_t rows, int cols, int fmt) {
    if (rows <= 0 || cols <= 0 || cols % 128 != 0 || !fmt_ok(fmt)) return 0;
    return cdiv(rows, 128) * 128 * (cols / (fmt == MOE_FP4_NV ? 16 : 32));
}

extern "C" int moe_quantize_rows_fp4(const moe_bf16* X, const moe_bf16* X1, const int64_t* rows_limit,
                                     int64_t rows, int cols, int fmt, uint8_t* Q, uint8_t* S, float* g,
                                     moe_stream_t stream) {
    if (!X || !Q || !S || !fmt_ok(fmt) || !g_ok(fmt, g)) return MOE_ERR_INVALID_ARG;
    if (rows <= 0 || cols <= 0) return MOE_ERR_INVALID_ARG;
    if (cols % 128 != 0 || (X1 ? 2 * (int64_t)cols : cols) > kFp4MaxCols) return MOE_ERR_UNSUPPORTED;
    if (!aligned16(X) || (X1 && !aligned16(X1)) || !aligned16(Q) || !aligned16(S) || !aligned4(g))
        return MOE_ERR_INVALID_ARG;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    return launch_quantize_rows_fp4(reinterpret_cast<const __nv_bfloat16*>(X),
                                    reinterpret_cast<const __nv_bfloat16*>(X1), rows_limit, rows, cols,
                                    fmt, Q, S, g, (cudaStream_t)stream);
}

extern "C" int moe_quantize_cols_fp4(const moe_bf16* X0, const moe_bf16* X1, int E, int K0, int N,
                                     int fmt, uint8_t* Qt, uint8_t* S, float* g, moe_stream_t stream) {
    if (!X0 || !Qt || !S || !fmt_ok(fmt) || !g_ok(fmt, g)) return MOE_ERR_INVALID_ARG;
    if (E <= 0 || K0 <= 0 || N <= 0) return MOE_ERR_INVALID_ARG;
    if (K0 % 128 != 0 || N % 128 != 0 || K0 > kFp4MaxCols || N > kFp4MaxCols || E > 65535)
        return MOE_ERR_UNSUPPORTED;
    if (!aligned16(X0) || (X1 && !aligned16(X1)) || !aligned16(Qt) || !aligned16(S) || !aligned4(g))
        return MOE_ERR_INVALID_ARG;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    cudaStream_t st = (cudaStream_t)stream;
    const auto* x0 = reinterpret_cast<const __nv_bfloat16*>(X0);
    const auto* x1 = reinterpret_cast<const __nv_bfloat16*>(X1);
    const int K = X1 ? 2 * K0 : K0;
    if (fmt == MOE_FP4_MX)
        return launch_cols<false, 64>(x0, x1, E, K0, N, K, K < kStripRowsMx ? K : kStripRowsMx, Qt, S, nullptr,
                                      false, st);
    // short columns: as many of them as give the threads a piece each (NC / 2 * K / 32 pieces). 16.8 M
    // elements in columns of 256: 33 us in strips of 16, 23 of 32, 21 of 64; of 512: 25, 21 and 23; of
    // 768: 26, 26, 28; of 1024: 23, 27, 29. Longer ones (16 matrices, 1024 columns each): of 1280 31 in
    // strips of 16 and of 32, of 1536 44 and 40, of 2048 58 and 58, of 2560 58 and 70; there a strip takes 47
    // KB and more in 16 columns, and twice that leaves two CTAs an SM or one
    if (K <= 256) return launch_cols<true, 64>(x0, x1, E, K0, N, K, K, Qt, S, g, false, st);
    if (K <= 640) return launch_cols<true, 32>(x0, x1, E, K0, N, K, K, Qt, S, g, false, st);
    if (K <= kStripMaxK) return launch_cols<true, 16>(x0, x1, E, K0, N, K, K, Qt, S, g, false, st);
    const int64_t n = (int64_t)E * N;
    if (cudaMemsetAsync(g, 0, sizeof(float) * n, st) != cudaSuccess) return MOE_ERR_LAUNCH;
    column_top_kernel<<<dim3((unsigned)(N / 128), (unsigned)E, (unsigned)cdiv(K, kTopRows)), kThreads, 0, st>>>(
        x0, x1, K0, N, reinterpret_cast<uint32_t*>(g));
    column_g_kernel<<<(unsigned)cdiv(n, 256), 256, 0, st>>>(g, n);
    if (launch_status() != MOE_OK) return MOE_ERR_LAUNCH;
    return launch_cols<true, 16>(x0, x1, E, K0, N, K, kStripRowsNv, Qt, S, g, true, st);
}

extern "C" int moe_dequantize_fp4(const uint8_t* Q, const uint8_t* S, const float* g,
                                  const int64_t* rows_limit, int64_t rows, int cols, int fmt,
                                  moe_bf16* out, moe_stream_t stream) {
    if (!Q || !S || !out || !fmt_ok(fmt) || !g_ok(fmt, g)) return MOE_ERR_INVALID_ARG;
    if (rows <= 0 || cols <= 0) return MOE_ERR_INVALID_ARG;
    if (cols % 128 != 0) return MOE_ERR_UNSUPPORTED;
    if (!aligned16(Q) || !aligned16(S) || !aligned16(out) || !aligned4(g)) return MOE_ERR_INVALID_ARG;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    auto* o = reinterpret_cast<__nv_bfloat16*>(out);
    return fmt == MOE_FP4_NV
               ? launch_dequantize<true>(Q, S, g, rows_limit, rows, cols, o, (cudaStream_t)stream)
               : launch_dequantize<false>(Q, S, g, rows_limit, rows, cols, o, (cudaStream_t)stream);
}

extern "C" int moe_permute_fp4(const uint8_t* xq, const uint8_t* sx, const float* gx,
                               const int32_t* slot_to_row, const int32_t* perm_token,
                               const int64_t* row_offsets, int64_t T, int64_t rows, int d, int E,
                               int k, int fmt, uint8_t* Xq, uint8_t* sX, float* gX, moe_stream_t stream) {
    if (!xq || !sx || !slot_to_row || !perm_token || !row_offsets || !Xq || !sX || !fmt_ok(fmt) ||
        !g_ok(fmt, gx) || !g_ok(fmt, gX))
        return MOE_ERR_INVALID_ARG;
    if (T <= 0 || rows <= 0 || d <= 0 || E <= 0 || k <= 0) return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts || k > E || k > 32 || d % 128 != 0 || rows > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    if (!aligned16(xq) || !aligned16(sx) || !aligned16(Xq) || !aligned16(sX) || !aligned4(gx) ||
        !aligned4(gX))
        return MOE_ERR_INVALID_ARG;
    if (!device_supported()) return MOE_ERR_UNSUPPORTED;
    int* status = device_status_word();
    if (!status) return MOE_ERR_LAUNCH;
    cudaStream_t st = (cudaStream_t)stream;
    const int ktiles = d / (fmt == MOE_FP4_NV ? Fp4<true>::TILE_K : Fp4<false>::TILE_K);
    const int64_t token_ctas = cdiv(T, kThreads / 32);
    return launch_dependent(permute_kernel, dim3((unsigned)(token_ctas + (int64_t)E * kPadSplit)), dim3(kThreads),
                            0, st, xq, sx, gx, slot_to_row, perm_token, row_offsets, T, rows, d, k, ktiles,
                            token_ctas, Xq, sX, gX, status);
}
