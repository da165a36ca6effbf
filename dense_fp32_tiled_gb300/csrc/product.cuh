// product.cuh -- the tensor-core product under the layer operators of GB300
// (sm_103a): its kernel, its plans and its operands.
//
// The kernel computes out[t][f] = sum_k Q[t][k] P[f][k] for "tokens" t (rows
// of out) and "features" f (its columns), with P, the weight or the operand
// that owns the columns, on the 128 rows of the tensor core and Q on its
// columns.  The features lie on the lanes of tensor memory then: an epilogue
// thread owns one feature (its bias is one register), a warp stores 32
// neighbouring features of one token, and the tile can be as narrow in tokens
// as a decoding step needs (16) without idle rows.
//   forward   P = w (N features),  Q = x          reduction over K
//   dx        P = w (K features),  Q = dz         reduction over N
//   dw        P, Q = x, dz transposed              reduction over the rows
// Each operand is read in the order it is held in: K-major or MN-major (the
// transposed one) is a matter of box shape and descriptor, so no operand is
// ever transposed in memory.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <type_traits>
#include <utility>

#include "linear.h"
#include "linear_prep.cuh"
#include "linear_types.cuh"
#include "nvtx_range.cuh"
#include "tensor_core.cuh"

namespace product {

using lt::from_f;
using lt::to_f;

constexpr int BK = 64;                       // K of a tile: one 128-byte swizzle row of 16-bit values
constexpr int PROWS = 128;                   // features per CTA
constexpr int P_BYTES = PROWS * BK * 2;      // 16 KiB
constexpr int MN_BOX_BYTES = 64 * BK * 2;    // an MN-major box: 64 operand rows x 64 K
constexpr int MAX_STAGES = 12;
constexpr int SORTED_EXPERTS = 256;         // of more, sorting by rows would take longer than it saves
constexpr int TMEM_COLS = 512;
constexpr int MAX_SPLITS = 4;                // CTAs of a cluster that share a tile's K; 8 took longer wherever tried
constexpr int EPI_WARPS = 8;                 // warp w: tensor-memory lanes 32 (w % 4).., column half w / 4
constexpr int COPY_WARP = EPI_WARPS, MMA_WARP = EPI_WARPS + 1, TAIL_WARP = EPI_WARPS + 2;
constexpr int THREADS = (EPI_WARPS + 3) * 32;
constexpr int EPI_THREADS = EPI_WARPS * 32;
constexpr int SMEM_MAX = 227 * 1024;
// FP32: a stage holds one piece of both operands, and a K tile is the stages
// of the third, second and first pieces in a row.  Their six products that
// matter run small ones first, (3,1) (1,3) (2,2) (2,1) (1,2) (1,1), each piece
// copied once for all of its products and its stage free after the last of
// them.  The tensor core's accumulation truncates, with an error that grows
// with the number of additions, so after KBLK tiles of K the accumulator is
// added in FP32 registers with round-to-nearest and starts again from zero.
constexpr int PIECES = 3;
constexpr int PRODUCTS = 6;
constexpr int KBLK = 2;
// Logits under an exponential: an error of theirs is one of the same size in its share, and
// those of likely targets are large sums of one sign, cut off always the same way.  After
// every K tile (4096 x 32768 x 2048 1689 us for 1651): gradients of 2533 x 23936 x 128 are
// 7e-7 off instead of 3.5e-6, a matrix product of FP32 FMAs before the exponential 1.2e-6.
constexpr int LOGITS_KBLK = 1;
constexpr int F32_COLS = 112;  // accumulator columns per epilogue thread: tiles up to 224 tokens
// The 16-bit types' logits are added up in registers too, after each `block` of K tiles: of
// LOGITS_BLOCK at most, and of FEW_BLOCK where one tile holds all tokens of a LOG_SUM, which
// then waits for the vocabulary's bytes (one token of 32768 x 4096 in bf16: blocks of 8 tiles
// 47.0 us, 4 47.4, 2 48.2, 1 49.3, and its log sum 4.3, 2.0, 0.9 and 0.9 x 1e-7 off).  With 8 tiles
// 8192 x 65536 x 2048 takes about as long as with none (1204 us, gradient 4081 for 4058), with
// 4 it takes 1311 and 4175.  A target's logit is a sum of one sign, so that what is cut off adds up:
// of tokens that the model is sure of (p = 0.98, 512 x 4096 x 8192 in bf16) dx is 2.3e-3 off and of the
// median one 3.1e-3, in one block 3.3e-3 and 3.3e-2 (from FP32 sums 1.7e-3 and 2.9e-3).
constexpr int LOGITS_BLOCK = 8, FEW_BLOCK = 2;
constexpr int LOGITS_REGS = 128;

enum Mode { DENSE = 0, ROWS_BY_EXPERT = 1, K_BY_EXPERT = 2 };

// What becomes of a tile.
//   LAYER             out = act(product + bias) + residual
// and, for the loss of a head over a vocabulary, with its tokens as features
// (a thread of the epilogue then owns a token) and its vocabulary as tokens:
//   LOG_SUM           nothing is stored but, of each token, the maximum and the
//                     sum of exponentials of its part of the tile, and the
//                     value at its target
//   SOFTMAX_GRADIENT  out = a exp(product - lse) - g [target] (FP32: in pieces)
//   SCALED_SUM        out = alpha (product + acc), or acc += product
// The last three have no splits and no experts.
enum Epilogue { LAYER = 0, LOG_SUM = 1, SOFTMAX_GRADIENT = 2, SCALED_SUM = 3 };
struct Token {  // of SOFTMAX_GRADIENT
    float lse;  // 16-bit types: times log2(e)
    float a, g;
    int target;  // -1: none
};
struct Loss {
    // LOG_SUM
    float2 *parts;        // two per tile of the vocabulary: [2 * tile + half][token]
    const void *targets;  // 4 or 8 bytes each
    float *hit;
    int target_bytes;
    // SOFTMAX_GRADIENT: tokens, and where the piece of the vocabulary begins
    const Token *tokens;
    int begin;
    long long piece;      // elements between FP32's pieces in out
    // SCALED_SUM
    float *acc;           // T x F
    const float *alpha;
    int first, last;      // acc holds nothing yet; out is wanted
    int chunks;           // of K, each with a T x F of its own in acc (1: none)
};

struct Product {
    int T, F, K;              // K_BY_EXPERT: K = all rows, shared out by offsets
    int mode, E;
    const int *offsets;
    int bt;                   // tokens per tile (multiple of 16 * CG)
    int nt, nf;               // tiles in tokens (DENSE, K_BY_EXPERT) and in features
    int splits;               // CTAs of a cluster that share the K of a tile (CG = 1)
    int stages, stage_bytes, q_bytes;
    int p_bytes;              // the loss's epilogues: of P's tile that are copied (see few_rows)
    int block;                // of the 16-bit types' logits: K tiles that are added up in tensor memory
    int epi_offset, epi_bytes;  // the epilogue's buffers in dynamic shared memory, per warp
    int p_mn, q_mn;
    const void *bias, *residual;
    void *z, *out;
    long long ldr, ldz, ldo, out_expert;
    int act;
    int widths;               // see OUT_SHIFT
    // a bias gradient to add up from the chunks' column sums on the side (see column_sum)
    const float *sums;
    void *dbias;
    int sums_M, sums_N, sums_E;
    int order;                // ORDER_*
    unsigned *timeout_flag;
    Loss loss;
};
// A backward pass's two products need the same earlier kernels and not each
// other.  The first lets the second start once it has waited for those
// (ORDER_FIRST); the second takes the SMs that the first leaves or never had,
// and waits for it before it ends (ORDER_BESIDE), so that what follows in the
// stream still comes after both.
enum Order { ORDER_ALONE = 0, ORDER_FIRST = 1, ORDER_BESIDE = 2 };
// Bytes of an access that all rows of out, z and the residual allow (16, 4 or 2), in Product::widths.
constexpr int OUT_SHIFT = 0, Z_SHIFT = 8, RESIDUAL_SHIFT = 16;
struct Maps {
    CUtensorMap p, q;
};

// One output tile: expert e, tokens [t0, t_end), features from f0 (of this
// CTA), K tiles [k0, k1) of this CTA, the first at element kbase.
struct Tile {
    int e, t0, t_end, ft, k0, k1, kbase, k_rows;
    bool none;  // rows of no expert: zeros
};

// Experts' tables in shared memory: clamped first rows and, for
// ROWS_BY_EXPERT, the first tile of each (group E: the rows of no expert).
// K_BY_EXPERT: the experts in falling order of rows.
struct Tables {
    const int *begin;  // E + 2
    const int *first;  // E + 2
};

// The unit's tile after idx: the same place in the next round of `units` tiles,
// or, where tiles come in falling order of length, back and forth, so that no
// unit always gets the longer ones.
__device__ __forceinline__ int next_tile(int idx, int unit, int units, bool snake) {
    if (!snake) return idx + units;
    const int round = idx / units;
    return (round + 1) * units + ((round & 1) == 0 ? units - 1 - unit : unit);
}
// Tile idx of nt x nf, 8 token tiles at a time: the tiles in flight share few
// panels of both operands.  Divisions only where they are needed: the first
// tile's copies wait for this.
__device__ __forceinline__ void raster(int idx, int nt, int nf, int &tt, int &ft) {
    int g = 0, r = idx;
    if (nt > 8) {
        const int per_group = 8 * nf;
        g = idx / per_group;
        r = idx - g * per_group;
    }
    const int rows = min(8, nt - 8 * g);
    if (rows == 8) {
        ft = r >> 3;
    } else if (rows == 1) {
        ft = r;
    } else {
        ft = r / rows;
    }
    tt = 8 * g + r - ft * rows;
}

// The same value, known to the compiler as one for the whole warp: what the
// issue loops derive from it stays in uniform registers.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// CHUNKS: tile idx of p.chunks * nt x nf, chunk e of K.
template <int CG, bool CHUNKS = false>
__device__ __forceinline__ Tile locate(int idx, const Product &p, const Tables &tb, int rank) {
    Tile w;
    int tt, ft, ktiles = (p.K + BK - 1) / BK;
    w.none = false;
    w.e = 0;
    w.kbase = 0;
    w.k_rows = p.K;
    if (p.mode == DENSE) {
        if (CHUNKS && p.loss.chunks > 1) {
            w.e = idx / (p.nt * p.nf);
            idx -= w.e * (p.nt * p.nf);
        }
        raster(idx, p.nt, p.nf, tt, ft);
        w.t0 = tt * p.bt;
        w.t_end = p.T;
    } else if (p.mode == ROWS_BY_EXPERT) {
        int lo = 0, hi = p.E + 1;  // the last group whose first tile is <= idx
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tb.first[mid] <= idx)
                lo = mid;
            else
                hi = mid;
        }
        w.e = lo;
        const int b = tb.begin[lo], n = tb.begin[lo + 1] - b;
        raster(idx - tb.first[lo], (n + p.bt - 1) / p.bt, p.nf, tt, ft);
        w.t0 = b + tt * p.bt;
        w.t_end = b + n;
        if (lo == p.E) {
            w.none = true;
            ktiles = 0;
        }
    } else {
        const int per = p.nt * p.nf;
        const int at = idx / per;
        w.e = tb.first[at];
        raster(idx - at * per, p.nt, p.nf, tt, ft);
        w.t0 = tt * p.bt;
        w.t_end = p.T;
        w.kbase = tb.begin[w.e];
        w.k_rows = tb.begin[w.e + 1] - w.kbase;
        ktiles = (w.k_rows + BK - 1) / BK;
    }
    if (p.mode != DENSE) {
        w.e = uniform(w.e);
        w.t0 = uniform(w.t0);
        w.t_end = uniform(w.t_end);
        ft = uniform(ft);
        w.kbase = uniform(w.kbase);
        w.k_rows = uniform(w.k_rows);
        ktiles = uniform(ktiles);
    }
    w.ft = ft;
    if (CG == 1 && p.splits > 1) {
        w.k0 = static_cast<int>(static_cast<long long>(ktiles) * rank / p.splits);
        w.k1 = static_cast<int>(static_cast<long long>(ktiles) * (rank + 1) / p.splits);
    } else if (CHUNKS && p.loss.chunks > 1) {
        w.k0 = static_cast<int>(static_cast<long long>(ktiles) * w.e / p.loss.chunks);
        w.k1 = static_cast<int>(static_cast<long long>(ktiles) * (w.e + 1) / p.loss.chunks);
    } else {
        w.k0 = 0;
        w.k1 = ktiles;
    }
    return w;
}

__device__ __forceinline__ void epi_bar() { asm volatile("bar.sync 1, %0;\n" ::"n"(EPI_THREADS) : "memory"); }

// Bias, activation, residual and the stores for 16 tokens (rows row0 .. of
// out, n of them valid) of one feature.
template <typename T>
__device__ __forceinline__ void finish16(const float (&acc)[16], const Product &p, float bias, int f, long long row0,
                                         int n, T *out, bool none) {
    constexpr bool EXACT = std::is_same<T, float>::value;
    if (n <= 0) return;
    T *o = out + row0 * p.ldo + f;
    if (none) {
        T *z = p.z != nullptr ? static_cast<T *>(p.z) + row0 * p.ldz + f : nullptr;
#pragma unroll
        for (int c = 0; c < 16; ++c)
            if (c < n) {
                o[c * p.ldo] = from_f<T>(0.0f);
                if (z != nullptr) z[c * p.ldz] = from_f<T>(0.0f);
            }
        return;
    }
    T r[16];
    const bool res = p.residual != nullptr;
    if (res) {
        const T *rp = static_cast<const T *>(p.residual) + row0 * p.ldr + f;
#pragma unroll
        for (int c = 0; c < 16; ++c)
            if (c < n) r[c] = rp[c * p.ldr];
    }
    float v[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) v[c] = acc[c] + bias;
    if (p.z != nullptr) {
        T *z = static_cast<T *>(p.z) + row0 * p.ldz + f;
#pragma unroll
        for (int c = 0; c < 16; ++c)
            if (c < n) z[c * p.ldz] = from_f<T>(v[c]);
    }
    lt::with_activation(p.act, [&](auto a) {
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] = lt::activate<decltype(a)::value, EXACT>(v[c]);
    });
    if (res) {
#pragma unroll
        for (int c = 0; c < 16; ++c)
            if (c < n) v[c] += to_f(r[c]);
    }
#pragma unroll
    for (int c = 0; c < 16; ++c)
        if (c < n) o[c * p.ldo] = from_f<T>(v[c]);
}

// ---- the 16-bit types' epilogue ------------------------------------------------
// A warp takes 32 features (the lanes of tensor memory that it may read) and 32
// tokens at a time, as 8 x 8 fragments.  A token's 32 features are 64
// contiguous bytes of out, so the fragments go through shared memory,
// transposed on the way by stmatrix, and leave in 16-byte stores, 8 tokens an
// instruction; the residual comes in the same way, copied ahead by cp.async
// while the tile is still being multiplied.  A row of the buffer is 64 bytes,
// its four 16-byte chunks XORed with half the row number, so that the eight
// rows of a matrix fall on different banks.
constexpr int EPI_T = 32;                      // tokens of a step
constexpr int STAGE16 = EPI_T * 64;            // bytes of a step's 32 x 32 values
// per warp: out, z, and two buffers of the residual
inline int epi_bytes(bool z, bool residual) { return STAGE16 * (1 + (z ? 1 : 0) + (residual ? 2 : 0)); }

__device__ __forceinline__ uint32_t stage16(uint32_t buf, int row, int chunk) {
    return buf + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}
// Rows that allow no 16-byte access move in narrower ones, 4 bytes if they can,
// but always with the lanes along the row: two rows or one an instruction.
// (Eight 2-byte stores of each lane's 16 bytes touch 32 rows' sectors each:
// 6783 x 1417 x 256 in bf16 with residual and saved argument took 117 us, so 60.)
// The rows' functions for narrow accesses are calls of their own: inlined, they cost the epilogue registers.
template <typename T>
__device__ __noinline__ void fetch_narrow(const T *base, long long ld, int F, int width, uint32_t buf, int n, int f0, int lane) {
    if (width == 4) {
        const int col = (lane & 15) * 2, f = f0 + col;
#pragma unroll 4
        for (int row = lane >> 4; row < n && row < EPI_T; row += 2) {
            const T *src = base + row * ld + col;
            const uint32_t dst = stage16(buf, row, col >> 3) + 2 * (col & 7);
            if (f + 1 < F)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
            else if (f < F)
                asm volatile("st.shared.b16 [%0], %1;\n" ::"r"(dst), "h"(*reinterpret_cast<const unsigned short *>(src)) : "memory");
        }
    } else {  // no asynchronous copy moves 2 bytes: 16 rows' loads together, then their stores
        const bool in = f0 + lane < F;
        const unsigned short *src = reinterpret_cast<const unsigned short *>(base) + lane;
#pragma unroll
        for (int h = 0; h < EPI_T; h += 16) {
            unsigned short v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = in && h + i < n ? src[(h + i) * ld] : static_cast<unsigned short>(0);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                asm volatile("st.shared.b16 [%0], %1;\n" ::"r"(stage16(buf, h + i, lane >> 3) + 2 * (lane & 7)), "h"(v[i])
                             : "memory");
        }
    }
}
// Residual rows row0 .. row0 + n of features f0 .. f0 + 31 into a buffer.
template <typename T>
__device__ __forceinline__ void fetch16(const Product &p, uint32_t buf, long long row0, int n, int f0, int lane) {
    const int width = (p.widths >> RESIDUAL_SHIFT) & 255;
    const T *base = static_cast<const T *>(p.residual) + row0 * p.ldr + f0;
    if (width == 16) {
#pragma unroll
        for (int i = 0; i < EPI_T / 8; ++i) {
            const int row = (lane >> 2) + 8 * i, chunk = lane & 3, f = f0 + 8 * chunk;
            if (row < n && f < p.F) {
                const T *src = base + row * p.ldr + 8 * chunk;
                const uint32_t dst = stage16(buf, row, chunk);
                if (f + 8 <= p.F) {
                    tc::cp_async16(dst, src);
                } else {
                    for (int k = 0; k < 8 && f + k < p.F; ++k)
                        asm volatile("st.shared.b16 [%0], %1;\n" ::"r"(dst + 2 * k),
                                     "h"(*reinterpret_cast<const unsigned short *>(src + k))
                                     : "memory");
                }
            }
        }
    } else {
        fetch_narrow<T>(base, p.ldr, p.F, width, buf, n, f0, lane);
    }
    tc::cp_async_commit();
}
// Asks for the residual of a warp's n tokens in L2 one tile ahead: from HBM it
// would arrive long after the step before has been finished.
template <typename T>
__device__ __forceinline__ void prefetch_residual(const Product &p, long long row0, int n, int f0, int lane) {
    const char *base = reinterpret_cast<const char *>(static_cast<const T *>(p.residual) + row0 * p.ldr + f0);
    for (int r = lane; r < n; r += 32)
        asm volatile("prefetch.global.L2 [%0];\n" ::"l"(base + r * p.ldr * static_cast<long long>(sizeof(T))) : "memory");
}
// The residual of the same warp's part of tile idx.
template <int CG, typename T>
__device__ __forceinline__ void prefetch_next(int idx, const Product &p, const Tables &tb, int rank, int col0, int cols, int lane0,
                                           int lane) {
    const Tile w = locate<CG>(idx, p, tb, rank);
    const int f0 = w.ft * (PROWS * CG) + (CG == 2 ? rank : 0) * PROWS + lane0;
    if (f0 < p.F && !w.none)
        prefetch_residual<T>(p, static_cast<long long>(w.t0) + col0, min(cols, min(p.bt, w.t_end - w.t0) - col0), f0, lane);
}
// 32 tokens x 32 features (fragments, rounded) into a buffer, and from there to
// rows row0 .. row0 + n of dst.
template <typename T>
__device__ __forceinline__ void stage_fragments(const float (&v)[2][16], uint32_t buf, int lane) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t r[4];
#pragma unroll
        for (int o = 0; o < 4; ++o) {
            const int i = 8 * (o >> 1) + 4 * (j & 1) + 2 * (o & 1);
            r[o] = lt::pack2<T>(v[j >> 1][i], v[j >> 1][i + 1]);
        }
        tc::stmatrix_t(stage16(buf, 8 * j + (lane & 7), lane >> 3), r);
    }
}
template <typename T>
__device__ __noinline__ void store_narrow(uint32_t buf, T *dst, long long ld, int width, int n, int f0, int F, int lane) {
    const int across = width == 4 ? 16 : 32, per = 32 / across;
    const int col = (lane & (across - 1)) * (32 / across), f = f0 + col;
    int row = width == 4 ? lane >> 4 : 0;
    T *o = dst + row * ld + col;
#pragma unroll 8
    for (; row < n && row < EPI_T; row += per, o += per * ld) {
        const uint32_t at = stage16(buf, row, col >> 3) + 2 * (col & 7);
        if (width == 4 && f + 1 < F) {
            uint32_t v;
            asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(v) : "r"(at) : "memory");
            *reinterpret_cast<uint32_t *>(o) = v;
        } else if (f < F) {
            unsigned short v;
            asm volatile("ld.shared.b16 %0, [%1];\n" : "=h"(v) : "r"(at) : "memory");
            *reinterpret_cast<unsigned short *>(o) = v;
        }
    }
}
template <typename T>
__device__ __forceinline__ void store_staged(uint32_t buf, T *dst, long long ld, int width, long long row0, int n, int f0,
                                             int F, int lane) {
    if (width == 16) {
        const int chunk = lane & 3, f = f0 + 8 * chunk;
        T *o = dst + (row0 + (lane >> 2)) * ld + f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t w[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                             : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                             : "r"(stage16(buf, (lane >> 2) + 8 * (2 * h + i), chunk))
                             : "memory");
#pragma unroll
            for (int i = 0; i < 2; ++i, o += 8 * ld) {
                if ((lane >> 2) + 8 * (2 * h + i) >= n || f >= F) continue;
                if (f + 8 <= F) {
                    *reinterpret_cast<uint4 *>(o) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (f + k < F)
                            reinterpret_cast<unsigned short *>(o)[k] = static_cast<unsigned short>(w[i][k >> 1] >> (16 * (k & 1)));
                }
            }
        }
    } else {
        store_narrow<T>(buf, dst + row0 * ld + f0, ld, width, n, f0, F, lane);
    }
}

// ---- the loss's epilogues --------------------------------------------------------
// log2(e) times what is left to the largest value: the difference first, as the
// product of each would lose what the largest has above the rest.
__device__ __forceinline__ float exp_of(float d) { return lt::fast_exp2(lt::kLog2E * d); }
__device__ __forceinline__ long long target_of(const Loss &l, int token) {
    return l.target_bytes == 8 ? static_cast<const long long *>(l.targets)[token]
                               : static_cast<long long>(static_cast<const int *>(l.targets)[token]);
}
// The running maximum and sum of exponentials of a token, 16 of its values (n of them valid) at a time.
struct LogSum {
    float high = -INFINITY, sum = 0.0f;
    __device__ __forceinline__ void add(float (&v)[16], int n) {
        if (n < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i >= n) v[i] = -INFINITY;
        }
        float m = high;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = fmaxf(m, v[i]);
        const float ref = m == -INFINITY ? 0.0f : m;  // -inf - -inf would be a NaN
        sum *= exp_of(high - ref);
        high = m;
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i & 3] += exp_of(v[i] - ref);
        sum += (s[0] + s[1]) + (s[2] + s[3]);
    }
};
// One tile of LOG_SUM, SOFTMAX_GRADIENT or SCALED_SUM, of this thread's lane of
// tensor memory: token (feature) f, columns col0 .. col0 + n of the tile.
// read(c, v) gives columns col0 + c .. col0 + c + 15.
template <typename T, int EPI, int COLS, typename Read>
__device__ __forceinline__ void loss_tile(const Product &p, const Tile &w, int f, bool f_ok, int col0, int n, Read &&read) {
    if constexpr (EPI == LOG_SUM) {
        LogSum ls;
        long long t = -1;
        if (f_ok) t = target_of(p.loss, f) - (static_cast<long long>(w.t0) + col0);
        const int at = t >= 0 && t < n ? static_cast<int>(t) : -1;
#pragma unroll
        for (int c = 0; c < COLS; c += 16)
            if (c < n) {
                float v[16];
                read(c, v);
                if ((at & ~15) == c) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c + i == at) p.loss.hit[f] = v[i];
                }
                ls.add(v, n - c);
            }
        const long long part = 2 * static_cast<long long>(w.t0 / p.bt) + (col0 != 0 ? 1 : 0);
        if (f_ok) p.loss.parts[part * p.F + f] = make_float2(ls.high, ls.sum);
    } else if constexpr (EPI == SOFTMAX_GRADIENT) {  // FP32; the 16-bit types' is below
        Token k = {0.0f, 0.0f, 0.0f, -1};
        if (f_ok) k = p.loss.tokens[f];
        const int t = k.target < 0 ? -1 : k.target - p.loss.begin - (w.t0 + col0);
#pragma unroll
        for (int c = 0; c < COLS; c += 16) {
            if (c >= n) break;
            float v[16];
            read(c, v);
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + (static_cast<long long>(w.t0) + col0 + c) * p.ldo + f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (c + i >= n || !f_ok) break;
                __nv_bfloat16 x, y, z;
                lt::pieces(fmaf(expf(v[i] - k.lse), k.a, c + i == t ? -k.g : 0.0f), x, y, z);
                o[i * p.ldo] = x;
                o[i * p.ldo + p.loss.piece] = y;
                o[i * p.ldo + 2 * p.loss.piece] = z;
            }
        }
    } else {
        const float alpha = p.loss.alpha != nullptr ? *p.loss.alpha : 1.0f;
        auto step = [&](int c) {
            float v[16], before[16];
            const long long row = static_cast<long long>(w.t0) + col0 + c;
            float *acc = p.loss.acc + (static_cast<long long>(w.e) * p.T + row) * p.F + f;
            if (!p.loss.first && f_ok) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c + i < n) before[i] = acc[static_cast<long long>(i) * p.F];
            }
            read(c, v);
            if (!f_ok) return;
            T *o = static_cast<T *>(p.out) + row * p.ldo + f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c + i < n) {
                    const float s = p.loss.first ? v[i] : v[i] + before[i];
                    if (p.loss.last)
                        o[i * p.ldo] = from_f<T>(s * alpha);
                    else
                        acc[static_cast<long long>(i) * p.F] = s;
                }
        };
        if constexpr (std::is_same<T, float>::value) {  // from registers, whose numbers are constants
#pragma unroll
            for (int c = 0; c < COLS; c += 16)
                if (c < n) step(c);
        } else {
            for (int c = 0; c < n; c += 16) step(c);
        }
    }
}

// SOFTMAX_GRADIENT of the 16-bit types, which rounds dz to them, as linear's gradient does
// its dz (dx and dw of 8192 x 65536 x 2048 in bf16 are then 1.8e-3 off and 1.7e-3 if only they
// are rounded, of 1003 x 5003 x 641 in float16 3.4e-4 and 2.9e-4; a second piece of dz would
// take both products twice), and their SCALED_SUM without acc where rows
// allow 16-byte accesses (narrower ones take longer through shared memory than straight
// from each lane: 960 x 40493 in bf16 80 us for 53): fragments through shared
// memory as in the layer's epilogue, four features a thread (8 o + lane / 4), so
// that rows of 32 leave in 16-byte stores.  release() is called when all accumulators
// have been read.  (Reading them one step ahead, as the layer's epilogue does, took
// longer here: 4346 x 43840 x 219 in bf16 143 us for 126.)
template <typename T, int EPI, typename Release>
__device__ __forceinline__ void staged_tile(const Product &p, const Tile &w, int f, bool f_ok, int col0, int n, bool any,
                                            uint32_t t_set, uint32_t buf, int lane, Release &&release) {
    if (n <= 0) {
        if (any) release();
        return;
    }
    const float alpha = EPI == SCALED_SUM ? *p.loss.alpha : 1.0f;
    Token mine = {0.0f, 0.0f, 0.0f, -1}, k[4];
    int t = -1;
    if constexpr (EPI == SOFTMAX_GRADIENT) {
        if (f_ok) mine = p.loss.tokens[f];
        t = mine.target < 0 ? -1 : mine.target - p.loss.begin - (w.t0 + col0);
        if (t < 0 || t >= n) t = -1;
#pragma unroll
        for (int o = 0; o < 4; ++o) {
            k[o].lse = __shfl_sync(0xffffffffu, mine.lse, 8 * o + (lane >> 2));
            k[o].a = __shfl_sync(0xffffffffu, mine.a, 8 * o + (lane >> 2));
            k[o].g = __shfl_sync(0xffffffffu, mine.g, 8 * o + (lane >> 2));
            k[o].target = __shfl_sync(0xffffffffu, t, 8 * o + (lane >> 2));
        }
    }
    const long long row0 = static_cast<long long>(w.t0) + col0;
    for (int c = 0; c < n; c += EPI_T) {
        float v[2][16];
        if (any) {
            tc::tmem_ld_frag(t_set + c, v[0]);
            tc::tmem_ld_frag(t_set + c + 16, v[1]);
            tc::tmem_ld_wait(v[0]);
            tc::tmem_ld_wait(v[1]);
            if (c + EPI_T >= n) release();
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 16; ++i) v[h][i] = 0.0f;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if constexpr (EPI == SCALED_SUM) {
                    v[h][i] *= alpha;
                } else {
                    const Token &q = k[2 * (i >> 3) + (i >> 1 & 1)];
                    v[h][i] = q.a * lt::fast_exp2(fmaf(v[h][i], lt::kLog2E, -q.lse));
                }
            }
        if constexpr (EPI == SOFTMAX_GRADIENT) {
            if (__any_sync(0xffffffffu, t >= c && t < c + EPI_T)) {  // a target among these
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const Token &q = k[2 * (i >> 3) + (i >> 1 & 1)];
                        if (q.target == c + 16 * h + 8 * (i >> 2 & 1) + 2 * (lane & 3) + (i & 1)) v[h][i] -= q.g;
                    }
            }
        }
        __syncwarp();  // the buffer's last contents have been read
        stage_fragments<T>(v, buf, lane);
        __syncwarp();
        store_staged<T>(buf, static_cast<T *>(p.out), p.ldo, (p.widths >> OUT_SHIFT) & 255, row0 + c, n - c, f - lane, p.F, lane);
    }
}

// A persistent grid of CTA pairs (CG = 2, tiles of 256 features) or of
// clusters of `splits` CTAs (CG = 1, 128 features, the K of a tile shared
// out).  Per CTA, warp 8 issues the tensor copies into a ring of stages, one
// K tile of P and Q each, warp 9 issues the products (in a pair, CTA 0's for
// both), warps 0-7 drain the accumulators, of which tensor memory holds two
// sets, while the next tile (FP32: the next block of K) is multiplied.
//
// Barriers: full[s] (of CTA 0 in a pair) completes when the copies of stage s
// have landed; empty[s] when the products reading it are done; acc_full[b]
// when accumulator set b is complete; acc_empty[b] (CTA 0) when all warps
// have read it; tail: see below; part_ready, part_read: the splits' hand-over.
//
// K_BY_EXPERT: the last K tile of an expert also holds rows of the next one.
// It is copied on a barrier of its own, tail_bar[s], and warp 10 clears those
// rows in both operands (a NaN times 0 would be one) and then reports the stage
// full, while the copies go on.  Before that, the same warp adds up the bias
// gradient, where the product is the first of a backward pass.
//
// MANY: a SOFTMAX_GRADIENT of the 16-bit types with more than one block of K: their sum goes back
// into tensor memory, from where it is read as the only one's is.  (A kernel of its own: the only
// block's needs 101 registers, this one 166.)
template <int CG, typename T, int EPI = LAYER, bool MANY = false>
__global__ void __launch_bounds__(THREADS, 1)
product_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Product p) {
    constexpr bool F32 = std::is_same<T, float>::value;
    constexpr bool BF16 = !std::is_same<T, __half>::value;  // FP32's pieces are bf16
    constexpr bool BLOCKS = F32 || EPI == LOG_SUM;          // K in blocks, added up in registers
    constexpr int COLS = F32 ? F32_COLS : LOGITS_REGS;
    const int block = !F32 ? p.block : EPI == LOG_SUM || EPI == SOFTMAX_GRADIENT ? LOGITS_KBLK : KBLK;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[MAX_STAGES], empty_bar[MAX_STAGES], acc_full[2], acc_empty[2];
    __shared__ __align__(8) uint64_t tail_bar[MAX_STAGES], part_ready, part_read;
    __shared__ uint32_t tmem_slot;
    const uint32_t sbase = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *sgen = smem_raw + (sbase - tc::smem_u32(smem_raw));
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t rank = uniform(static_cast<int>(tc::cluster_rank()));
    const int S = CG == 1 ? p.splits : 1;
    const int cluster = CG == 2 ? 2 : S;
    const int unit = blockIdx.x / cluster, units = gridDim.x / cluster;
    const uint32_t lead = CG == 2 ? 0 : rank;
    float *partial = reinterpret_cast<float *>(sgen + static_cast<size_t>(p.stages) * p.stage_bytes);
    int *tables = reinterpret_cast<int *>(partial + (S > 1 ? p.bt * PROWS : 0));
    const Tables tb{tables, tables + p.E + 2};
    // P's tile in a stage; Q's follows it
    const uint32_t p_bytes = EPI == LOG_SUM || EPI == SOFTMAX_GRADIENT ? p.p_bytes : P_BYTES;
    const uint32_t epi = tc::smem_u32(smem_raw) + p.epi_offset + (warp < EPI_WARPS ? warp : 0) * p.epi_bytes;

    if (warp == 0) {  // a barrier or three per lane: one thread would take as long as a copy from L2
        if (lane < p.stages) {
            tc::mbar_init(tc::smem_u32(&full_bar[lane]), CG);
            tc::mbar_init(tc::smem_u32(&empty_bar[lane]), 1);
            tc::mbar_init(tc::smem_u32(&tail_bar[lane]), 1);
        } else if (lane < MAX_STAGES + 2) {
            const int b = lane - MAX_STAGES;
            if (b >= 0) {
                tc::mbar_init(tc::smem_u32(&acc_full[b]), 1);
                tc::mbar_init(tc::smem_u32(&acc_empty[b]), CG * EPI_WARPS);
            }
        } else if (lane == MAX_STAGES + 2) {
            tc::mbar_init(tc::smem_u32(&part_ready), S);
            tc::mbar_init(tc::smem_u32(&part_read), S);
        }
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    } else if (warp == COPY_WARP && lane == 0) {
        tc::tma_prefetch(&maps.p);
        tc::tma_prefetch(&maps.q);
    }
    // nothing of global memory is touched before the earlier kernels are done
    if (p.order != ORDER_BESIDE) tc::grid_wait();
    if (p.order == ORDER_FIRST) tc::grid_trigger();
    int tiles = p.nt * p.nf;
    if (p.mode != DENSE) {
        // clamp: non-decreasing and inside the rows, whatever the offsets hold
        const int rows = p.mode == ROWS_BY_EXPERT ? p.T : p.K;
        if (warp == 0) {
            int high = 0, tile0 = 0;
            for (int e0 = 0; e0 < p.E + 2; e0 += 32) {
                const int e = e0 + lane;
                int b = rows > 0 && e <= p.E ? min(max(p.offsets[e], 0), rows) : rows;  // without rows there may be no offsets
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xffffffffu, b, d);
                    if (lane >= d) b = max(b, o);
                }
                b = max(b, high);
                if (e < p.E + 2) tables[e] = b;
                high = __shfl_sync(0xffffffffu, b, 31);
            }
            __syncwarp();
            if (p.mode == K_BY_EXPERT) {
                for (int e = lane; e < p.E; e += 32) {
                    int at = e;
                    if (p.E <= SORTED_EXPERTS) {
                        const int n = tables[e + 1] - tables[e];
                        at = 0;
                        for (int o = 0; o < p.E; ++o) {
                            const int m = tables[o + 1] - tables[o];
                            at += m > n || (m == n && o < e) ? 1 : 0;
                        }
                    }
                    tables[p.E + 2 + at] = e;
                }
            } else
                for (int e0 = 0; e0 < p.E + 2; e0 += 32) {
                    const int e = e0 + lane;
                    const int n = e <= p.E ? (tables[e + 1] - tables[e] + p.bt - 1) / p.bt * p.nf : 0;
                    int sum = n;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const int o = __shfl_up_sync(0xffffffffu, sum, d);
                        if (lane >= d) sum += o;
                    }
                    if (e < p.E + 2) tables[p.E + 2 + e] = tile0 + sum - n;
                    tile0 += __shfl_sync(0xffffffffu, sum, 31);
                }
        }
    }
    __syncthreads();
    tc::cluster_sync();  // the barriers of all CTAs exist before any remote arrive or copy
    // the first copies are on their way while tensor memory is allocated
    uint32_t tmem = 0;
    if (warp < EPI_WARPS || warp == MMA_WARP) {
        if (warp == MMA_WARP) tc::tmem_alloc<CG, TMEM_COLS>(tc::smem_u32(&tmem_slot));
        tc::fence_before();
        asm volatile("bar.sync 2, %0;\n" ::"n"(EPI_THREADS + 32) : "memory");
        tc::fence_after();
        tmem = uniform(static_cast<int>(tmem_slot));
    }
    if (EPI == SCALED_SUM) tiles *= p.loss.chunks;
    if (p.mode == ROWS_BY_EXPERT)
        tiles = tb.first[p.E + 1];
    else if (p.mode == K_BY_EXPERT)
        tiles *= p.E;
    const bool snake = p.mode == K_BY_EXPERT;
    tc::Waiter waiter(p.timeout_flag);

    // One thread issues the copies and one the products, so what they run per
    // stage is kept to the least: no divisions, the stage and its phase counted along.
    const int q_rows = p.bt / CG;
    const uint32_t stage_bytes = p.stage_bytes;
    const int stages = p.stages;
    if (warp == COPY_WARP) {
        const uint32_t full0 = CG == 2 ? tc::peer_addr(tc::smem_u32(&full_bar[0]), 0) : tc::smem_u32(&full_bar[0]);
        const uint32_t empty0 = tc::smem_u32(&empty_bar[0]);
        const uint32_t tail0 = CG == 2 ? tc::peer_addr(tc::smem_u32(&tail_bar[0]), rank) : tc::smem_u32(&tail_bar[0]);
        const uint32_t bytes = p_bytes + p.q_bytes;
        const bool p_mn = p.p_mn != 0, q_mn = p.q_mn != 0;
        const int z_planes = p.mode == ROWS_BY_EXPERT ? p.E : 1;
        uint32_t ph = 1;
        int s = 0, issued = 0;  // stage; how many of the ring are in use, at most
        for (int idx = unit; idx < tiles; idx = next_tile(idx, unit, units, snake)) {
            const Tile w = locate<CG, EPI == SCALED_SUM>(idx, p, tb, static_cast<int>(rank));
            const int f0 = w.ft * (PROWS * CG) + static_cast<int>(CG == 2 ? rank : 0) * PROWS;
            const int tq = w.t0 + static_cast<int>(CG == 2 ? rank : 0) * q_rows;
            const int z_p = p.mode == ROWS_BY_EXPERT ? w.e : 0;
            // of K_BY_EXPERT: the K tile that also holds the next expert's rows
            const int tail_kt = p.mode == K_BY_EXPERT && w.k_rows % BK != 0 ? w.k_rows / BK : -1;
            int k = w.kbase + w.k0 * BK;
            for (int kt = w.k0; kt < w.k1; ++kt, k += BK) {
                const bool tail = kt == tail_kt;
#pragma unroll
                for (int piece = F32 ? PIECES - 1 : 0; piece >= 0; --piece) {
                    const int zp = z_p + piece * z_planes, zq = piece;
                    const uint32_t st = sbase + s * stage_bytes;
                    waiter.wait(empty0 + 8u * s, ph);  // passes at once on a ring not yet used
                    __syncwarp();
                    if (tc::elect()) {
                        const uint32_t bar = (tail ? tail0 : full0) + 8u * s;
                        tc::mbar_arrive_expect<CG>(bar, bytes);
                        if (p_mn) {
                            tc::tma_load_3d<CG>(st, &maps.p, f0, k, zp, bar);
                            tc::tma_load_3d<CG>(st + MN_BOX_BYTES, &maps.p, f0 + 64, k, zp, bar);
                        } else {
                            tc::tma_load_3d<CG>(st, &maps.p, k, f0, zp, bar);
                        }
                        if (q_mn) {
                            for (int i = 0; i < q_rows; i += 64)
                                tc::tma_load_3d<CG>(st + p_bytes + i * (MN_BOX_BYTES / 64), &maps.q, tq + i, k, zq, bar);
                        } else {
                            tc::tma_load_3d<CG>(st + p_bytes, &maps.q, k, tq, zq, bar);
                        }
                    }
                    __syncwarp();
                    issued = min(issued + 1, stages);
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
        }
        // this CTA's last copies are read before it can exit; after a wait that ran out, they
        // are given one more limit to land
        waiter.gave_up = false;
        for (; issued > 0; --issued) {
            if (s == 0) {
                s = stages;
                ph ^= 1;
            }
            --s;
            waiter.wait(empty0 + 8u * s, ph ^ 1);
        }
    } else if (warp == TAIL_WARP) {
        if (p.dbias != nullptr) {
            const int strips = (p.sums_N + 31) / 32;
            const long long jobs = static_cast<long long>(strips) * (p.sums_E < 0 ? 1 : p.sums_E);
            for (long long j = blockIdx.x; j < jobs; j += gridDim.x) {
                const int e = static_cast<int>(j / strips), col = static_cast<int>(j - static_cast<long long>(e) * strips) * 32 + lane;
                const float t = linear_prep::column_sum(p.sums, p.sums_M, p.sums_N, p.sums_E, p.offsets, e, col, 0, 1);
                if (col < p.sums_N) static_cast<T *>(p.dbias)[static_cast<long long>(e) * p.sums_N + col] = from_f<T>(t);
            }
        }
        if (p.mode == K_BY_EXPERT) {
            const uint32_t full0 = tc::peer_addr(tc::smem_u32(&full_bar[0]), lead);
            const int boxes = (P_BYTES + p.q_bytes) / MN_BOX_BYTES;
            uint32_t phases = 0;  // of tail_bar, a bit per stage
            int s = 0;
            for (int idx = unit; idx < tiles; idx = next_tile(idx, unit, units, snake)) {
                const Tile w = locate<CG, EPI == SCALED_SUM>(idx, p, tb, static_cast<int>(rank));
                const int left = w.k_rows % BK;  // both operands are MN-major: a box row is one K
                const bool tail = left != 0 && w.k0 <= w.k_rows / BK && w.k_rows / BK < w.k1;
                s = (s + (F32 ? PIECES : 1) * (w.k1 - w.k0 - (tail ? 1 : 0))) % stages;
                if (!tail) continue;
                for (int piece = 0; piece < (F32 ? PIECES : 1); ++piece) {
                    waiter.wait(tc::smem_u32(&tail_bar[s]), (phases >> s) & 1);
                    phases ^= 1u << s;
                    const int chunks = (BK - left) * 8;  // 16-byte chunks to clear in each box
                    uint8_t *sg = sgen + static_cast<size_t>(s) * stage_bytes + left * 128;
                    for (int b = 0; b < boxes; ++b)
                        for (int i = lane; i < chunks; i += 32)
                            *reinterpret_cast<uint4 *>(sg + b * MN_BOX_BYTES + i * 16) = make_uint4(0, 0, 0, 0);
                    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(full0 + 8u * s);
                    if (++s == stages) s = 0;
                }
            }
        }
    } else if (warp == MMA_WARP) {
        if (rank == lead) {
            const uint32_t idesc = tc::instr_desc_f16(BF16, p.p_mn != 0, p.q_mn != 0, PROWS * CG, p.bt);
            const uint32_t p_step = (p.p_mn ? 2048u : 32u) >> 4, q_step = (p.q_mn ? 2048u : 32u) >> 4;  // per 16 K
            const uint64_t ad0 = tc::smem_desc(sbase, p.p_mn ? MN_BOX_BYTES : 16);
            const uint64_t bd0 = tc::smem_desc(sbase + p_bytes, p.q_mn ? MN_BOX_BYTES : 16);
            const uint32_t full0 = tc::smem_u32(&full_bar[0]), empty0 = tc::smem_u32(&empty_bar[0]);
            uint32_t ph = 0, g = 0;
            int s = 0;
            for (int idx = unit; idx < tiles; idx = next_tile(idx, unit, units, snake)) {
                const Tile w = locate<CG, EPI == SCALED_SUM>(idx, p, tb, static_cast<int>(rank));
                const int tail_kt = p.mode == K_BY_EXPERT && w.k_rows % BK != 0 ? w.k_rows / BK : -1;
                for (int kb = w.k0; kb < w.k1; kb += BLOCKS || MANY ? block : w.k1 - w.k0, ++g) {
                    const int ke = BLOCKS || MANY ? min(kb + block, w.k1) : w.k1;
                    const uint32_t set = g & 1;
                    waiter.wait(tc::smem_u32(&acc_empty[set]), ((g >> 1) & 1) ^ 1);
                    tc::fence_after();
                    const uint32_t d = tmem + set * (TMEM_COLS / 2);
                    uint32_t more = 0;
                    // 64 K of the operands in two stages (P's and Q's), as four instructions
                    auto multiply = [&](int sp, int sq) {
                        const uint64_t ad = ad0 + ((sp * stage_bytes) >> 4), bd = bd0 + ((sq * stage_bytes) >> 4);
#pragma unroll
                        for (int j = 0; j < BK / 16; ++j)
                            tc::umma_f16<CG>(d, ad + j * p_step, bd + j * q_step, idesc, j > 0 ? 1u : more);
                        more = 1;
                    };
                    auto advance = [&] {
                        if (++s == stages) {
                            s = 0;
                            ph ^= 1;
                        }
                    };
                    for (int kt = kb; kt < ke; ++kt) {
                        int third = 0, second = 0;
                        if constexpr (F32) {
                            waiter.wait(full0 + 8u * s, ph);
                            third = s;
                            advance();
                            waiter.wait(full0 + 8u * s, ph);
                            second = s;
                            advance();
                        }
                        if (kt == tail_kt)  // with rows that the tail warps cleared, here and in the other CTA
                            waiter.wait<true>(full0 + 8u * s, ph);
                        else
                            waiter.wait(full0 + 8u * s, ph);
                        tc::fence_after();
                        __syncwarp();
                        if (tc::elect()) {
                            if constexpr (F32) {
                                multiply(third, s);
                                multiply(s, third);
                                tc::umma_commit<CG>(empty0 + 8u * third);
                                multiply(second, second);
                                multiply(second, s);
                                multiply(s, second);
                                tc::umma_commit<CG>(empty0 + 8u * second);
                            }
                            multiply(s, s);
                            tc::umma_commit<CG>(empty0 + 8u * s);
                        }
                        more = 1;
                        advance();
                    }
                    __syncwarp();
                    if (tc::elect()) tc::umma_commit<CG>(tc::smem_u32(&acc_full[set]));
                }
            }
        }
    } else {
        const int q = warp & 3, h = warp >> 2;
        const int half = p.bt >= 32 ? p.bt / 2 : 16;
        const int col0 = h * half;                  // this warp's columns: [col0, col0 + cols)
        const int cols = min(half, p.bt - col0);
        const uint32_t t_off = (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(col0);
        const uint32_t acc_empty0 = tc::peer_addr(tc::smem_u32(&acc_empty[0]), lead);
        uint32_t g = 0, handed = 0;
        for (int idx = unit; idx < tiles; idx = next_tile(idx, unit, units, snake)) {
            const Tile w = locate<CG, EPI == SCALED_SUM>(idx, p, tb, static_cast<int>(rank));
            const int fl = 32 * q + lane;           // feature within the CTA's 128
            const int f = w.ft * (PROWS * CG) + static_cast<int>(CG == 2 ? rank : 0) * PROWS + fl;
            T *out = static_cast<T *>(p.out) + (p.mode == K_BY_EXPERT ? w.e * p.out_expert : 0);
            const int n_tile = min(p.bt, w.t_end - w.t0);
            const bool f_ok = f < p.F;
            float bias = 0.0f;
            if (p.bias != nullptr && f_ok && !w.none)
                bias = to_f(static_cast<const T *>(p.bias)[(p.mode == ROWS_BY_EXPERT ? static_cast<long long>(w.e) * p.F : 0) + f]);
            const bool any = w.k1 > w.k0;
            float total[BLOCKS || MANY ? COLS : 1];
            if constexpr (MANY) {
#pragma unroll
                for (int c = 0; c < COLS; ++c) total[c] = 0.0f;
                for (int kb = w.k0; kb < w.k1; kb += block) {
                    const uint32_t set = g & 1;
                    waiter.wait(tc::smem_u32(&acc_full[set]), (g / 2) & 1);
                    __syncwarp();
                    tc::fence_after();
                    const uint32_t t_set = tmem + set * (TMEM_COLS / 2) + t_off;
                    const bool last = kb + block >= w.k1;
#pragma unroll
                    for (int c = 0; c < COLS; c += 16)
                        if (c < cols) {
                            float v[16];
                            tc::tmem_ld16(t_set + c, v);
                            tc::tmem_ld_wait(v);
#pragma unroll
                            for (int i = 0; i < 16; ++i) total[c + i] += v[i];
                            if (last) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) v[i] = total[c + i];
                                tc::tmem_st16(t_set + c, v);
                            }
                        }
                    if (last) break;  // its set is reported read where the sum is
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive_relaxed(acc_empty0 + 8u * set);
                    ++g;
                }
                tc::tmem_st_wait();
            }
            if constexpr (BLOCKS) {
                if (p.residual != nullptr && !w.none && S == 1 && f - lane < p.F)
                    prefetch_residual<T>(p, static_cast<long long>(w.t0) + col0, min(cols, n_tile - col0), f - lane, lane);
#pragma unroll
                for (int c = 0; c < COLS; ++c) total[c] = 0.0f;
                for (int kb = w.k0; kb < w.k1; kb += block, ++g) {
                    const uint32_t set = g & 1;
                    waiter.wait(tc::smem_u32(&acc_full[set]), (g / 2) & 1);
                    __syncwarp();
                    tc::fence_after();
                    const uint32_t t_set = tmem + set * (TMEM_COLS / 2) + t_off;
#pragma unroll
                    for (int c = 0; c < COLS; c += 16)
                        if (c < cols) {
                            float v[16];
                            tc::tmem_ld16(t_set + c, v);
                            tc::tmem_ld_wait(v);
#pragma unroll
                            for (int i = 0; i < 16; ++i) total[c + i] += v[i];
                        }
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive_relaxed(acc_empty0 + 8u * set);
                }
            }
            const uint32_t set = g & 1;
            bool freed = false;  // the accumulators are reported read
            const uint32_t t_set = tmem + set * (TMEM_COLS / 2) + t_off;
            if constexpr (EPI != LAYER) {
                const int n = f - lane < p.F ? min(cols, n_tile - col0) : 0;
                if (!BLOCKS && any) {
                    waiter.wait(tc::smem_u32(&acc_full[set]), (g / 2) & 1);
                    __syncwarp();
                    tc::fence_after();
                }
                bool done = false;
                if constexpr (!F32 && EPI != LOG_SUM) {
                    if (EPI == SOFTMAX_GRADIENT || (p.loss.first && p.loss.last && ((p.widths >> OUT_SHIFT) & 255) == 16)) {
                        staged_tile<T, EPI>(p, w, f, f_ok, col0, n, any, t_set, epi, lane, [&] {
                            tc::fence_before();
                            __syncwarp();
                            if (lane == 0) tc::mbar_arrive_relaxed(acc_empty0 + 8u * set);
                        });
                        done = true;
                    }
                }
                if (!done) {
                    auto read = [&](int c, float (&v)[16]) {
                        if constexpr (BLOCKS) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] = total[c + i];  // c is a constant there
                        } else if (any) {
                            __syncwarp();  // the loads are the whole warp's
                            tc::tmem_ld16(t_set + c, v);
                            tc::tmem_ld_wait(v);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] = 0.0f;
                        }
                    };
                    loss_tile<T, EPI, COLS>(p, w, f, f_ok, col0, n, read);
                }
                if (!BLOCKS && any) {
                    if (!done) {
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive_relaxed(acc_empty0 + 8u * set);
                    }
                    ++g;
                }
                continue;
            }
            if (S > 1 && !w.none) {
                // hand this CTA's part over: wait until the last one is read, store, tell all
                if (handed > 0) waiter.wait<true>(tc::smem_u32(&part_read), (handed - 1) & 1);
                if (!F32 && any) {
                    waiter.wait(tc::smem_u32(&acc_full[set]), (g / 2) & 1);
                    __syncwarp();
                    tc::fence_after();
                }
#pragma unroll
                for (int c = 0; c < 64; c += 16)  // split tiles have at most 128 tokens
                    if (c < cols) {
                        float v[16];
                        if constexpr (F32) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] = total[c + i];
                        } else if (any) {
                            tc::tmem_ld16(t_set + c, v);
                            tc::tmem_ld_wait(v);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] = 0.0f;
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) partial[(col0 + c + i) * PROWS + fl] = v[i];
                    }
                asm volatile("fence.acq_rel.cluster;\n" ::: "memory");
            } else if constexpr (F32) {
#pragma unroll
                for (int c = 0; c < F32_COLS; c += 16)
                    if (c < cols && f_ok && (S == 1 || rank == 0)) {
                        float v[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = total[c + i];
                        finish16<T>(v, p, bias, f, static_cast<long long>(w.t0) + col0 + c, n_tile - (col0 + c), out, w.none);
                    }
            } else if (S == 1 || rank == 0) {
                const int f0 = f - lane;
                const int n_warp = f0 < p.F ? min(cols, n_tile - col0) : 0;  // this warp's tokens
                const long long row0 = static_cast<long long>(w.t0) + col0;
                float b[4];
#pragma unroll
                for (int o = 0; o < 4; ++o) b[o] = __shfl_sync(0xffffffffu, bias, 8 * o + (lane >> 2));
                const bool res = p.residual != nullptr && !w.none;
                const uint32_t obuf = epi, zbuf = epi + STAGE16, rbuf0 = epi + (p.z != nullptr ? 2 : 1) * STAGE16;
                if (res && n_warp > 0) {
                    fetch16<T>(p, rbuf0, row0, n_warp, f0, lane);
                    if (idx == unit && n_warp > EPI_T) prefetch_residual<T>(p, row0 + EPI_T, n_warp - EPI_T, f0, lane);
                }
                if (any) {
                    waiter.wait(tc::smem_u32(&acc_full[set]), (g / 2) & 1);
                    __syncwarp();
                    tc::fence_after();
                }
                float next[2][16];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 16; ++i) next[h][i] = 0.0f;
                if (any && n_warp > 0) {
                    tc::tmem_ld_frag(t_set, next[0]);
                    tc::tmem_ld_frag(t_set + 16, next[1]);
                    tc::tmem_ld_wait(next[0]);
                    tc::tmem_ld_wait(next[1]);
                }
                if (p.residual != nullptr && next_tile(idx, unit, units, snake) < tiles)
                    prefetch_next<CG, T>(next_tile(idx, unit, units, snake), p, tb, static_cast<int>(rank), col0, cols, 32 * q, lane);
                for (int c = 0; c < n_warp; c += EPI_T) {
                    const uint32_t rbuf = rbuf0 + (c / EPI_T & 1) * STAGE16;
                    if (res) {  // the next step's residual, into the buffer read last time
                        __syncwarp();
                        if (c + EPI_T < n_warp)
                            fetch16<T>(p, rbuf0 + ((c / EPI_T & 1) ^ 1) * STAGE16, row0 + c + EPI_T, n_warp - c - EPI_T, f0, lane);
                    }
                    float v[2][16];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[h][i] = next[h][i];
                    const bool more = any && c + EPI_T < n_warp;
                    if (more) {  // arrives while these are finished
                        tc::tmem_ld_frag(t_set + c + EPI_T, next[0]);
                        tc::tmem_ld_frag(t_set + c + EPI_T + 16, next[1]);
                    } else if (any) {  // all read: the accumulators are free while the rest is finished
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive_relaxed(acc_empty0 + 8u * set);
                        freed = true;
                    }
                    __syncwarp();  // the buffers' last contents have been read
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[h][i] += b[2 * (i >> 3) + (i >> 1 & 1)];
                    if (p.z != nullptr) stage_fragments<T>(v, zbuf, lane);
                    if (!w.none)
                        lt::with_activation(p.act, [&](auto a) {
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int i = 0; i < 16; ++i) v[h][i] = lt::activate<decltype(a)::value, F32>(v[h][i]);
                        });
                    if (res) {
                        if (c + EPI_T < n_warp)
                            tc::cp_async_wait<1>();
                        else
                            tc::cp_async_wait<0>();
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t r[4];
                            tc::ldmatrix_t(stage16(rbuf, 8 * j + (lane & 7), lane >> 3), r);
#pragma unroll
                            for (int o = 0; o < 4; ++o) {
                                const int i = 8 * (o >> 1) + 4 * (j & 1) + 2 * (o & 1);
                                const float2 x = lt::unpack2<T>(r[o]);
                                v[j >> 1][i] += x.x;
                                v[j >> 1][i + 1] += x.y;
                            }
                        }
                    }
                    stage_fragments<T>(v, obuf, lane);
                    __syncwarp();
                    if (p.z != nullptr)
                        store_staged<T>(zbuf, static_cast<T *>(p.z), p.ldz, (p.widths >> Z_SHIFT) & 255, row0 + c, n_warp - c, f0, p.F, lane);
                    store_staged<T>(obuf, out, p.ldo, (p.widths >> OUT_SHIFT) & 255, row0 + c, n_warp - c, f0, p.F, lane);
                    if (more) {
                        tc::tmem_ld_wait(next[0]);
                        tc::tmem_ld_wait(next[1]);
                    }
                }
            }
            if (!F32 && any) {
                if (!freed) {
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive_relaxed(acc_empty0 + 8u * set);
                }
                ++g;
            }
            if (S > 1 && !w.none) {
                epi_bar();
                if (threadIdx.x < S) tc::mbar_arrive(tc::peer_addr(tc::smem_u32(&part_ready), threadIdx.x));
                waiter.wait<true>(tc::smem_u32(&part_ready), handed & 1);
                // the parts' sum in rank order, four features of a token per thread, shared out over
                // all CTAs, two such at a time with their loads in flight together
                const uint32_t mine = tc::smem_u32(partial);
                const int fb = w.ft * PROWS;
                const T *bias_e = p.bias == nullptr ? nullptr
                                                    : static_cast<const T *>(p.bias) +
                                                          (p.mode == ROWS_BY_EXPERT ? static_cast<long long>(w.e) * p.F : 0);
                constexpr int U = 2;
                const int items = n_tile * (PROWS / 4), step = S * EPI_THREADS;
                for (int i0 = static_cast<int>(rank) * EPI_THREADS + threadIdx.x; i0 < items; i0 += U * step) {
                    float4 part[U][MAX_SPLITS];
                    float b[U][4], r[U][4];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int i = i0 + u * step, fi = fb + 4 * (i & (PROWS / 4 - 1));
                        const bool in = i < items && fi < p.F;
#pragma unroll
                        for (int s = 0; s < MAX_SPLITS; ++s)
                            part[u][s] = in && s < S ? tc::ld_cluster_f32x4(tc::peer_addr(mine + 16u * i, s)) : make_float4(0, 0, 0, 0);
                        const T *rp = static_cast<const T *>(p.residual) +
                                      (static_cast<long long>(w.t0) + i / (PROWS / 4)) * p.ldr + fi;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const bool ok = in && fi + k < p.F;
                            b[u][k] = ok && bias_e != nullptr ? to_f(bias_e[fi + k]) : 0.0f;
                            r[u][k] = ok && p.residual != nullptr ? to_f(rp[k]) : 0.0f;
                        }
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int i = i0 + u * step, fi = fb + 4 * (i & (PROWS / 4 - 1));
                        if (i >= items || fi >= p.F) continue;
                        const long long row = static_cast<long long>(w.t0) + i / (PROWS / 4);
                        float v[4] = {part[u][0].x, part[u][0].y, part[u][0].z, part[u][0].w};
#pragma unroll
                        for (int s = 1; s < MAX_SPLITS; ++s)
                            v[0] += part[u][s].x, v[1] += part[u][s].y, v[2] += part[u][s].z, v[3] += part[u][s].w;
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] += b[u][k];
                        if (p.z != nullptr) {
                            T *z = static_cast<T *>(p.z) + row * p.ldz + fi;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (fi + k < p.F) z[k] = from_f<T>(v[k]);
                        }
                        lt::with_activation(p.act, [&](auto a) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) v[k] = lt::activate<decltype(a)::value, F32>(v[k]);
                        });
                        T *o = out + row * p.ldo + fi;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (fi + k < p.F) o[k] = from_f<T>(p.residual != nullptr ? v[k] + r[u][k] : v[k]);
                    }
                }
                epi_bar();
                if (threadIdx.x < S) tc::mbar_arrive(tc::peer_addr(tc::smem_u32(&part_read), threadIdx.x));
                ++handed;
            }
        }
    }
    if (p.order == ORDER_BESIDE) tc::grid_wait();
    tc::fence_before();
    __syncthreads();
    tc::cluster_sync();  // no remote arrive and no read of this CTA's memory is still pending
    if (warp == MMA_WARP) tc::tmem_free<CG, TMEM_COLS>(tmem);
}

// ---- host: set-up ----------------------------------------------------------------
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiledFn encode_fn() {
    static EncodeTiledFn found = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            found = reinterpret_cast<EncodeTiledFn>(fn);
        else
            (void)cudaGetLastError();
    });
    return found;
}

struct Device {
    int state = 0;  // 0 not set up, 1 ready, < 0 a status
    unsigned long long ctx = 0;
    int sms = 0, pairs = 0;
    unsigned *timeout_flag = nullptr;
};

// ---- host: one product --------------------------------------------------------------
// An operand as the tensor copies see it: `outer` rows of `inner` 16-bit
// values, `planes` of them.
struct Operand {
    const void *base = nullptr;
    long long inner = 0, outer = 0, planes = 1;
    long long ld = 0, plane = 0;  // elements
    bool mn = false;              // inner runs along the operand's rows (else along K)
};

inline bool encode(CUtensorMap &map, const Operand &o, bool f16, int box_outer) {
    const cuuint64_t dim[3] = {static_cast<cuuint64_t>(o.inner), static_cast<cuuint64_t>(o.outer),
                               static_cast<cuuint64_t>(o.planes)};
    const long long plane = o.planes > 1 ? o.plane : o.ld * o.outer;
    const cuuint64_t stride[2] = {static_cast<cuuint64_t>(o.ld) * 2, static_cast<cuuint64_t>(plane) * 2};
    const cuuint32_t box[3] = {BK, static_cast<cuuint32_t>(box_outer), 1};
    const cuuint32_t ones[3] = {1, 1, 1};
    return encode_fn()(&map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                       const_cast<void *>(o.base), dim, stride, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Narrowest tile of LOG_SUM, T x F: the room for its parts is known without a plan.
// Only products of few tiles want one narrower than 128.
inline int log_sum_columns(long long T, long long F) { return T * F > 1 << 22 ? 128 : 64; }
struct Plan {
    int cg = 2, bt = 256, splits = 1, units = 1;
    double cost = 1e300;
};

// LINEAR_TUNE="cg=1|2,bt=16..256,splits=1..4", read once at the first call,
// limits the plans of every product to those values, for sweeps without a
// rebuild.  Limits that leave a product no plan are not applied to it, and the
// first time that is said on stderr.  It changes how the work is split, not
// what is computed.
struct Tune {
    int cg = 0, bt = 0, splits = 0;
};
inline const Tune &tune() {
    static const Tune t = [] {
        Tune r;
        const char *env = std::getenv("LINEAR_TUNE");
        while (env != nullptr && *env != 0) {
            if (strncmp(env, "cg=", 3) == 0) r.cg = std::atoi(env + 3);
            if (strncmp(env, "bt=", 3) == 0) r.bt = std::atoi(env + 3);
            if (strncmp(env, "splits=", 7) == 0) r.splits = std::atoi(env + 7);
            const char *next = strchr(env, ',');
            env = next != nullptr ? next + 1 : nullptr;
        }
        return r;
    }();
    return t;
}

// Bytes of Q's tile: rows of 64 K, or whole boxes of 64 rows (the last one, of
// which fewer may be wanted, is copied whole).
inline int q_bytes_of(int rows, bool mn) { return mn ? (rows + 63) / 64 * MN_BOX_BYTES : rows * 128; }

// Time of a plan in SM clocks.  A K tile of a CTA (128 features, bt tokens, 64
// K; FP32: three stages of pieces) takes the longest of three: the tensor cores' bt/2 clocks per 16 K (2.2 bt
// measured for the four with bt = 256), the bytes that it copies at what L2
// gives an SM when all copy (62 a clock measured), and the issue of a stage
// (370 clocks measured with narrow tiles).  Whole waves of tiles count, and
// between filling the pipeline and draining the last accumulator about 6000
// clocks pass.  Measured on 4096^3 in bf16 (us): pairs 224 wide 73, 256 wide 82,
// 128 wide 95; single CTAs 256 wide 93, 128 wide 126.
inline Plan choose(const Product &p, const Device &d, int type, const Tune &only, int least = 0, int chunks = 1) {
    const bool f32 = type == LINEAR_F32;
    Plan best;
    const int bts[] = {256, 224, 192, 160, 128, 96, 64, 32, 16};
    for (int cg = 2; cg >= 1; --cg)
        for (int bt : bts) {
            if (bt < least || (cg == 2 && (bt < 64 || bt % 32 != 0))) continue;
            if (f32 && bt > 2 * F32_COLS) continue;
            if ((only.cg != 0 && only.cg != cg) || (only.bt != 0 && only.bt != bt)) continue;
            double nt, ktiles = (p.K + BK - 1) / BK;
            if (p.mode == ROWS_BY_EXPERT) {
                // the host does not know the counts: as if the rows were spread evenly
                const double met = p.E < p.T ? p.E : p.T;
                const double each = met > 0 ? p.T / met : 0;
                nt = met * (each <= bt ? 1.0 : each / bt + 0.5);
            } else {
                nt = (p.T + bt - 1) / bt;
                if (p.mode == K_BY_EXPERT) {
                    nt *= p.E;
                    ktiles = (p.K / (p.E > 0 ? p.E : 1) + BK - 1) / BK + 0.5;
                }
            }
            nt *= chunks;
            ktiles /= chunks;
            const double tiles = nt * ((p.F + PROWS * cg - 1) / (PROWS * cg));
            double per = 370.0;
            const double copy = (P_BYTES + q_bytes_of(bt / cg, p.q_mn != 0)) / 62.0;
            if (copy > per) per = copy;
            if (f32) per *= PIECES;
            const double mma = (f32 ? PRODUCTS : 1) * 2.2 * bt;
            if (mma > per) per = mma;
            const double drain = 1000.0 + 12.0 * bt;
            const int most = cg == 2 || bt > 128 ? 1 : MAX_SPLITS;
            for (int s = 1; s <= most; ++s) {
                if (s > 1 && s * 2 > ktiles) break;
                if (only.splits != 0 && only.splits != s) continue;
                const int units = cg == 2 ? d.pairs : d.sms / s;
                double waves = static_cast<double>(static_cast<long long>((tiles + units - 1) / units));
                if (waves < 1) waves = 1;
                if (s > 1 && waves > 1 && only.splits == 0) break;  // a split is for fewer tiles than SMs
                const double body = ktiles / s * per + 200.0;
                const double cost = waves * (body > drain ? body : drain) + drain + (s > 1 ? 1500.0 + 45.0 * bt : 0.0) + 2000.0;
                if (cost < best.cost * 0.99) {
                    best.cost = cost;
                    best.cg = cg;
                    best.bt = bt;
                    best.splits = s;
                    best.units = units;
                }
            }
        }
    return best;
}

// Rows of P's tile that are copied.  A copy takes as long for a row outside the
// operand as for one inside (one token of 32768 x 4096 in bf16: 64 us), so of
// few tokens only theirs are copied; the tensor core then takes what lies behind them
// in the stage for the tile's other rows, which come out on lanes that nothing reads.
inline int few_rows(const Product &p, int epi, const Plan &pl, const Operand &P) {
    if ((epi != LOG_SUM && epi != SOFTMAX_GRADIENT) || P.mn || pl.cg != 1 || p.F >= PROWS) return PROWS;
    return (p.F + 7) / 8 * 8;
}

template <int CG, typename T, int EPI, bool MANY>
cudaError_t launch(const Maps &maps, const Product &p, int grid, size_t smem, cudaStream_t stream) {
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG == 2 ? 2 : static_cast<unsigned>(p.splits);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, product_kernel<CG, T, EPI, MANY>, maps, p);
}

// Enqueue one product: P and Q as 16-bit operands (FP32: three planes each).
template <int EPI>
int run_product(int type, Product p, const Operand &P, const Operand &Q, const Device &d, cudaStream_t stream,
                int *token_tiles = nullptr, int *chunks = nullptr) {
    if (p.T == 0 || p.F == 0 || (p.mode == K_BY_EXPERT && p.E == 0)) return SGEMM_OK;
    p.p_mn = P.mn;
    p.q_mn = Q.mn;
    p.timeout_flag = d.timeout_flag;
    Tune only = tune();
    if (EPI != LAYER) only.splits = 1;
    const int least = EPI == LOG_SUM ? log_sum_columns(p.T, p.F) : 0;
    if (only.bt < least) only.bt = 0;  // no narrower ones
    Plan pl = choose(p, d, type, only, least);
    if (pl.cost > 1e299) {
        static std::once_flag told;
        std::call_once(told, [&] {
            fprintf(stderr, "LINEAR_TUNE leaves no plan for a product of %d x %d x %d and is not applied to it\n", p.T, p.F, p.K);
        });
        only = Tune();
        if (EPI != LAYER) only.splits = 1;
        pl = choose(p, d, type, only, least);
    }
    p.loss.chunks = 1;
    if (EPI == SCALED_SUM && chunks != nullptr) {
        const int ktiles = (p.K + BK - 1) / BK;
        if (*chunks >= 0) {  // as many as the piece before had
            p.loss.chunks = *chunks;
            pl = choose(p, d, type, only, 0, *chunks);
        } else {
            // of few tiles and a long K, shares of it side by side; joining them takes 4 us and
            // what they write and read
            for (int c = 2; c <= -*chunks && 4 * c <= ktiles; c += (c + 3) / 4) {
                Plan with = choose(p, d, type, only, 0, c);
                with.cost += 8000.0 + static_cast<double>(c) * p.T * p.F * 8 / (d.sms * 20.0);
                if (with.cost < 0.9 * pl.cost) {
                    pl = with;
                    p.loss.chunks = c;
                }
            }
            *chunks = p.loss.chunks;
        }
        if (*chunks > 1) p.loss.last = 0;
    }
    p.bt = pl.bt;
    p.splits = pl.splits;
    p.q_bytes = q_bytes_of(p.bt / pl.cg, Q.mn);
    const int p_rows = few_rows(p, EPI, pl, P);
    p.p_bytes = p_rows * 128;
    // blocks of K as long as one another
    const int ktiles = (p.K + BK - 1) / BK, most = EPI == LOG_SUM && p.F <= PROWS ? FEW_BLOCK : LOGITS_BLOCK;
    const int blocks = (ktiles + most - 1) / most;
    p.block = blocks > 0 ? (ktiles + blocks - 1) / blocks : 1;
    p.stage_bytes = p.p_bytes + p.q_bytes;
    if (p.stage_bytes < P_BYTES) p.stage_bytes = P_BYTES;
    const int per_unit = PROWS * pl.cg;
    p.nf = (p.F + per_unit - 1) / per_unit;
    p.nt = (p.T + p.bt - 1) / p.bt;
    if (token_tiles != nullptr) *token_tiles = p.nt;
    long long tiles = static_cast<long long>(p.nt) * p.nf;
    if (p.mode == ROWS_BY_EXPERT) tiles = (static_cast<long long>(p.nt) + p.E + 1) * p.nf;  // at most
    if (p.mode == K_BY_EXPERT) tiles *= p.E;
    tiles *= p.loss.chunks;
    if (tiles > INT_MAX / 2) return SGEMM_ERR_INVALID_DIM;
    const int tables = p.mode == DENSE ? 0 : 2 * (p.E + 2) * 4;
    const int part = p.splits > 1 ? p.bt * PROWS * 4 : 0;
    p.epi_bytes = epi_bytes(p.z != nullptr, p.residual != nullptr && p.splits == 1);  // split: only zero rows go there
    const int epi = type == LINEAR_F32 ? 0 : EPI_WARPS * p.epi_bytes + 128;
    p.stages = (SMEM_MAX - 2048 - tables - part - epi) / p.stage_bytes;
    if (p.stages > MAX_STAGES) p.stages = MAX_STAGES;
    const size_t used = 1024 + static_cast<size_t>(p.stages) * p.stage_bytes + part + tables;
    p.epi_offset = static_cast<int>((used + 127) / 128 * 128);
    const size_t smem = used + epi;
    auto width = [&](const void *base, long long ld, long long expert) {
        const unsigned long long bits = reinterpret_cast<uintptr_t>(base) | static_cast<unsigned long long>(ld | expert) * 2;
        return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
    };
    p.widths = width(p.out, p.ldo, p.out_expert) << OUT_SHIFT | width(p.z, p.ldz, 0) << Z_SHIFT |
               width(p.residual, p.ldr, 0) << RESIDUAL_SHIFT;
    Maps maps;
    memset(&maps, 0, sizeof maps);
    const bool f16 = type == LINEAR_F16;
    if (p.K > 0 && (!encode(maps.p, P, f16, P.mn ? BK : p_rows) || !encode(maps.q, Q, f16, Q.mn ? BK : p.bt / pl.cg)))
        return SGEMM_ERR_DEVICE;
    const int units = static_cast<int>(tiles < pl.units ? tiles : pl.units);
    const int grid = units * (pl.cg == 2 ? 2 : p.splits);
    sg_nvtx::Range r("linear: product");
    auto start = [&](auto el, auto many) {
        using El = decltype(el);
        constexpr bool MANY = decltype(many)::value;
        return pl.cg == 2 ? launch<2, El, EPI, MANY>(maps, p, grid, smem, stream) : launch<1, El, EPI, MANY>(maps, p, grid, smem, stream);
    };
    auto half = [&](auto el) {
        if constexpr (EPI == SOFTMAX_GRADIENT)
            if (blocks > 1) return start(el, std::true_type());
        return start(el, std::false_type());
    };
    const cudaError_t err = type == LINEAR_F32    ? start(float(), std::false_type())
                            : type == LINEAR_BF16 ? half(__nv_bfloat16())
                                                  : half(__half());
    if (err != cudaSuccess) {
        (void)cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    return SGEMM_OK;
}

// ---- host: operands -------------------------------------------------------------------
inline size_t up256(long long bytes) { return (static_cast<size_t>(bytes) + 255) / 256 * 256; }
inline long long up8(long long n) { return (n + 7) / 8 * 8; }

// A matrix (or E of them) of the call: `outer` rows of `inner` values.
struct Matrix {
    const void *base = nullptr;
    long long inner = 0, outer = 0, planes = 1;
    long long ld = 0, plane = 0;
};

// Whether the tensor copies can read it as it is: 16-bit values, 16-byte
// aligned rows.
inline bool direct(int type, const Matrix &m) {
    return type != LINEAR_F32 && reinterpret_cast<uintptr_t>(m.base) % 16 == 0 && m.ld % 8 == 0 &&
           (m.planes <= 1 || m.plane % 8 == 0);
}
inline long long copy_elements(const Matrix &m) { return m.planes * m.outer * up8(m.inner); }
// Workspace of the operand: nothing, an aligned copy, or the three FP32 pieces.
inline size_t operand_bytes(int type, const Matrix &m) {
    if (m.inner <= 0 || m.outer <= 0 || m.planes <= 0 || direct(type, m)) return 0;
    return up256(copy_elements(m) * 2 * (type == LINEAR_F32 ? 3 : 1));
}
// The operands of a call that need a copy: laid out in the workspace one after
// the other, and made in one launch.
struct Copies {
    linear_prep::Copy list[2];
    int n = 0;
    char *ws;
    explicit Copies(char *workspace) : ws(workspace) {}

    Operand operand(int type, const Matrix &m, bool mn) {
        Operand o;
        o.mn = mn;
        o.inner = m.inner;
        o.outer = m.outer;
        o.planes = m.planes;
        if (m.inner <= 0 || m.outer <= 0 || m.planes <= 0) return o;
        if (direct(type, m)) {
            o.base = m.base;
            o.ld = m.ld;
            o.plane = m.plane;
            return o;
        }
        o.base = ws;
        o.ld = up8(m.inner);
        o.plane = m.outer * o.ld;
        if (type == LINEAR_F32) o.planes *= PIECES;
        list[n++] = linear_prep::Copy{m.base, m.ld, m.plane, static_cast<int>(m.inner), static_cast<int>(m.outer),
                                      static_cast<int>(m.planes), ws};
        ws += operand_bytes(type, m);
        return o;
    }
    int run(int type, cudaStream_t stream) {
        if (linear_prep::copy_operands(type, list, n, stream) == cudaSuccess) return SGEMM_OK;
        (void)cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
};

// ---- host: argument checks ---------------------------------------------------------------
struct Span {
    uintptr_t lo = 0, hi = 0;
};
inline Span span(const void *p, long long rows, long long width, long long ld, int bytes) {
    Span s;
    if (p == nullptr || rows <= 0 || width <= 0) return s;
    s.lo = reinterpret_cast<uintptr_t>(p);
    s.hi = s.lo + static_cast<uintptr_t>(((rows - 1) * ld + width) * bytes);
    return s;
}
inline bool overlap(const Span &a, const Span &b) { return a.lo < b.hi && b.lo < a.hi; }
inline bool misaligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }
inline long long at_least_1(long long v) { return v > 1 ? v : 1; }

inline Matrix row_matrix(const void *p, int rows, int width, long long ld) {
    Matrix m;
    m.base = p;
    m.inner = width;
    m.outer = rows;
    m.ld = ld;
    m.plane = rows * ld;
    return m;
}

// ---- in linear.cu ------------------------------------------------------------------------
// The current device's set-up, made at its first call.
int set_up(Device *out);
// A product with the layer's epilogue.
int run_layer(int type, const Product &p, const Operand &P, const Operand &Q, const Device &d, cudaStream_t stream);
// Allows this kernel all the shared memory that a product may use.
template <int CG, typename T, int EPI, bool MANY = false>
bool opt_in() {
    return cudaFuncSetAttribute(product_kernel<CG, T, EPI, MANY>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX - 1024) ==
           cudaSuccess;
}

}  // namespace product
