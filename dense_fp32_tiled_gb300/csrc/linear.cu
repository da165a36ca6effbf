// linear.cu -- the layer products of GB300 (sm_103a): y = act(x.w + bias) +
// residual, the same over rows grouped by expert, and the products of their
// gradients, all on one tensor-core kernel (C ABI: include/linear.h).
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
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <type_traits>
#include <utility>

#include "ctx_key.cuh"
#include "linear.h"
#include "linear_few.cuh"
#include "linear_prep.cuh"
#include "linear_types.cuh"
#include "nvtx_range.cuh"
#include "tensor_core.cuh"

namespace {

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
constexpr int F32_COLS = 112;  // accumulator columns per epilogue thread: tiles up to 224 tokens

enum Mode { DENSE = 0, ROWS_BY_EXPERT = 1, K_BY_EXPERT = 2 };

struct Product {
    int T, F, K;              // K_BY_EXPERT: K = all rows, shared out by offsets
    int mode, E;
    const int *offsets;
    int bt;                   // tokens per tile (multiple of 16 * CG)
    int nt, nf;               // tiles in tokens (DENSE, K_BY_EXPERT) and in features
    int splits;               // CTAs of a cluster that share the K of a tile (CG = 1)
    int stages, stage_bytes, q_bytes;
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

template <int CG>
__device__ __forceinline__ Tile locate(int idx, const Product &p, const Tables &tb, int rank) {
    Tile w;
    int tt, ft, ktiles = (p.K + BK - 1) / BK;
    w.none = false;
    w.e = 0;
    w.kbase = 0;
    w.k_rows = p.K;
    if (p.mode == DENSE) {
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
template <int CG, typename T>
__global__ void __launch_bounds__(THREADS, 1)
product_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Product p) {
    constexpr bool F32 = std::is_same<T, float>::value;
    constexpr bool BF16 = !std::is_same<T, __half>::value;  // FP32's pieces are bf16
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
        const uint32_t bytes = P_BYTES + p.q_bytes;
        const bool p_mn = p.p_mn != 0, q_mn = p.q_mn != 0;
        const int z_planes = p.mode == ROWS_BY_EXPERT ? p.E : 1;
        uint32_t ph = 1;
        int s = 0, issued = 0;  // stage; how many of the ring are in use, at most
        for (int idx = unit; idx < tiles; idx = next_tile(idx, unit, units, snake)) {
            const Tile w = locate<CG>(idx, p, tb, static_cast<int>(rank));
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
                                tc::tma_load_3d<CG>(st + P_BYTES + i * (MN_BOX_BYTES / 64), &maps.q, tq + i, k, zq, bar);
                        } else {
                            tc::tma_load_3d<CG>(st + P_BYTES, &maps.q, k, tq, zq, bar);
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
                const Tile w = locate<CG>(idx, p, tb, static_cast<int>(rank));
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
            const uint64_t bd0 = tc::smem_desc(sbase + P_BYTES, p.q_mn ? MN_BOX_BYTES : 16);
            const uint32_t full0 = tc::smem_u32(&full_bar[0]), empty0 = tc::smem_u32(&empty_bar[0]);
            uint32_t ph = 0, g = 0;
            int s = 0;
            for (int idx = unit; idx < tiles; idx = next_tile(idx, unit, units, snake)) {
                const Tile w = locate<CG>(idx, p, tb, static_cast<int>(rank));
                const int tail_kt = p.mode == K_BY_EXPERT && w.k_rows % BK != 0 ? w.k_rows / BK : -1;
                for (int kb = w.k0; kb < w.k1; kb += F32 ? KBLK : w.k1 - w.k0, ++g) {
                    const int ke = F32 ? min(kb + KBLK, w.k1) : w.k1;
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
            const Tile w = locate<CG>(idx, p, tb, static_cast<int>(rank));
            const int fl = 32 * q + lane;           // feature within the CTA's 128
            const int f = w.ft * (PROWS * CG) + static_cast<int>(CG == 2 ? rank : 0) * PROWS + fl;
            T *out = static_cast<T *>(p.out) + (p.mode == K_BY_EXPERT ? w.e * p.out_expert : 0);
            const int n_tile = min(p.bt, w.t_end - w.t0);
            const bool f_ok = f < p.F;
            float bias = 0.0f;
            if (p.bias != nullptr && f_ok && !w.none)
                bias = to_f(static_cast<const T *>(p.bias)[(p.mode == ROWS_BY_EXPERT ? static_cast<long long>(w.e) * p.F : 0) + f]);
            const bool any = w.k1 > w.k0;
            float total[F32 ? F32_COLS : 1];
            if constexpr (F32) {
                if (p.residual != nullptr && !w.none && S == 1 && f - lane < p.F)
                    prefetch_residual<T>(p, static_cast<long long>(w.t0) + col0, min(cols, n_tile - col0), f - lane, lane);
#pragma unroll
                for (int c = 0; c < F32_COLS; ++c) total[c] = 0.0f;
                for (int kb = w.k0; kb < w.k1; kb += KBLK, ++g) {
                    const uint32_t set = g & 1;
                    waiter.wait(tc::smem_u32(&acc_full[set]), (g / 2) & 1);
                    __syncwarp();
                    tc::fence_after();
                    const uint32_t t_set = tmem + set * (TMEM_COLS / 2) + t_off;
#pragma unroll
                    for (int c = 0; c < F32_COLS; c += 16)
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

__device__ unsigned g_linear_timeout;

// ---- host: set-up ----------------------------------------------------------------
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
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
std::mutex g_mutex;
Device g_devices[64];

template <int CG, typename T>
bool opt_in() {
    return cudaFuncSetAttribute(product_kernel<CG, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX - 1024) ==
           cudaSuccess;
}

int set_up(Device *out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return SGEMM_ERR_DEVICE;
    }
    if (dev < 0 || dev >= 64) return SGEMM_ERR_DEVICE;
    unsigned long long ctx = 0;
    const bool known = sg_ctx::current_id(dev, &ctx);
    std::lock_guard<std::mutex> lock(g_mutex);
    Device &d = g_devices[dev];
    if (known && d.state != 0 && d.ctx != ctx) d.state = 0;  // a new context
    if (d.state == 0) {
        d.ctx = ctx;
        int major = 0, minor = 0;
        int st = SGEMM_OK;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || major != 10 ||
            minor != 3 || d.sms < 2 || encode_fn() == nullptr || !opt_in<1, float>() || !opt_in<2, float>() ||
            !opt_in<1, __nv_bfloat16>() || !opt_in<2, __nv_bfloat16>() || !opt_in<1, __half>() ||
            !opt_in<2, __half>() ||
            cudaGetSymbolAddress(reinterpret_cast<void **>(&d.timeout_flag), g_linear_timeout) != cudaSuccess)
            st = SGEMM_ERR_DEVICE;
        d.pairs = d.sms / 2;
        if (st == SGEMM_OK) {
            cudaLaunchConfig_t cfg;
            memset(&cfg, 0, sizeof cfg);
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = 2;
            attr.val.clusterDim.y = 1;
            attr.val.clusterDim.z = 1;
            cfg.gridDim = dim3(static_cast<unsigned>(2 * d.pairs));
            cfg.blockDim = dim3(THREADS);
            cfg.dynamicSmemBytes = SMEM_MAX - 1024;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, product_kernel<2, __nv_bfloat16>, &cfg) == cudaSuccess && n > 0)
                d.pairs = n < d.pairs ? n : d.pairs;
        }
        (void)cudaGetLastError();
        d.state = st == SGEMM_OK ? 1 : st;
    }
    *out = d;
    return d.state > 0 ? SGEMM_OK : d.state;
}

// ---- host: one product --------------------------------------------------------------
// An operand as the tensor copies see it: `outer` rows of `inner` 16-bit
// values, `planes` of them.
struct Operand {
    const void *base = nullptr;
    long long inner = 0, outer = 0, planes = 1;
    long long ld = 0, plane = 0;  // elements
    bool mn = false;              // inner runs along the operand's rows (else along K)
};

bool encode(CUtensorMap &map, const Operand &o, bool f16, int box_outer) {
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
const Tune &tune() {
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
int q_bytes_of(int rows, bool mn) { return mn ? (rows + 63) / 64 * MN_BOX_BYTES : rows * 128; }

// Time of a plan in SM clocks.  A K tile of a CTA (128 features, bt tokens, 64
// K; FP32: three stages of pieces) takes the longest of three: the tensor cores' bt/2 clocks per 16 K (2.2 bt
// measured for the four with bt = 256), the bytes that it copies at what L2
// gives an SM when all copy (62 a clock measured), and the issue of a stage
// (370 clocks measured with narrow tiles).  Whole waves of tiles count, and
// between filling the pipeline and draining the last accumulator about 6000
// clocks pass.  Measured on 4096^3 in bf16 (us): pairs 224 wide 73, 256 wide 82,
// 128 wide 95; single CTAs 256 wide 93, 128 wide 126.
Plan choose(const Product &p, const Device &d, int type, const Tune &only) {
    const bool f32 = type == LINEAR_F32;
    Plan best;
    const int bts[] = {256, 224, 192, 160, 128, 96, 64, 32, 16};
    for (int cg = 2; cg >= 1; --cg)
        for (int bt : bts) {
            if (cg == 2 && (bt < 64 || bt % 32 != 0)) continue;
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

template <int CG, typename T>
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
    return cudaLaunchKernelEx(&cfg, product_kernel<CG, T>, maps, p);
}

// Enqueue one product: P and Q as 16-bit operands (FP32: three planes each).
int run_product(int type, Product p, const Operand &P, const Operand &Q, const Device &d, cudaStream_t stream) {
    if (p.T == 0 || p.F == 0 || (p.mode == K_BY_EXPERT && p.E == 0)) return SGEMM_OK;
    p.p_mn = P.mn;
    p.q_mn = Q.mn;
    p.timeout_flag = d.timeout_flag;
    Plan pl = choose(p, d, type, tune());
    if (pl.cost > 1e299) {
        static std::once_flag told;
        std::call_once(told, [&] {
            fprintf(stderr, "LINEAR_TUNE leaves no plan for a product of %d x %d x %d and is not applied to it\n", p.T, p.F, p.K);
        });
        pl = choose(p, d, type, Tune());
    }
    p.bt = pl.bt;
    p.splits = pl.splits;
    p.q_bytes = q_bytes_of(p.bt / pl.cg, Q.mn);
    p.stage_bytes = P_BYTES + p.q_bytes;
    const int per_unit = PROWS * pl.cg;
    p.nf = (p.F + per_unit - 1) / per_unit;
    p.nt = (p.T + p.bt - 1) / p.bt;
    long long tiles = static_cast<long long>(p.nt) * p.nf;
    if (p.mode == ROWS_BY_EXPERT) tiles = (static_cast<long long>(p.nt) + p.E + 1) * p.nf;  // at most
    if (p.mode == K_BY_EXPERT) tiles *= p.E;
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
    if (p.K > 0 && (!encode(maps.p, P, f16, P.mn ? BK : PROWS) || !encode(maps.q, Q, f16, Q.mn ? BK : p.bt / pl.cg)))
        return SGEMM_ERR_DEVICE;
    const int units = static_cast<int>(tiles < pl.units ? tiles : pl.units);
    const int grid = units * (pl.cg == 2 ? 2 : p.splits);
    sg_nvtx::Range r("linear: product");
    cudaError_t err;
    if (pl.cg == 2)
        err = type == LINEAR_F32    ? launch<2, float>(maps, p, grid, smem, stream)
              : type == LINEAR_BF16 ? launch<2, __nv_bfloat16>(maps, p, grid, smem, stream)
                                    : launch<2, __half>(maps, p, grid, smem, stream);
    else
        err = type == LINEAR_F32    ? launch<1, float>(maps, p, grid, smem, stream)
              : type == LINEAR_BF16 ? launch<1, __nv_bfloat16>(maps, p, grid, smem, stream)
                                    : launch<1, __half>(maps, p, grid, smem, stream);
    if (err != cudaSuccess) {
        (void)cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    return SGEMM_OK;
}

// ---- host: operands -------------------------------------------------------------------
size_t up256(long long bytes) { return (static_cast<size_t>(bytes) + 255) / 256 * 256; }
long long up8(long long n) { return (n + 7) / 8 * 8; }

// A matrix (or E of them) of the call: `outer` rows of `inner` values.
struct Matrix {
    const void *base = nullptr;
    long long inner = 0, outer = 0, planes = 1;
    long long ld = 0, plane = 0;
};

// Whether the tensor copies can read it as it is: 16-bit values, 16-byte
// aligned rows.
bool direct(int type, const Matrix &m) {
    return type != LINEAR_F32 && reinterpret_cast<uintptr_t>(m.base) % 16 == 0 && m.ld % 8 == 0 &&
           (m.planes <= 1 || m.plane % 8 == 0);
}
long long copy_elements(const Matrix &m) { return m.planes * m.outer * up8(m.inner); }
// Workspace of the operand: nothing, an aligned copy, or the three FP32 pieces.
size_t operand_bytes(int type, const Matrix &m) {
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
Span span(const void *p, long long rows, long long width, long long ld, int bytes) {
    Span s;
    if (p == nullptr || rows <= 0 || width <= 0) return s;
    s.lo = reinterpret_cast<uintptr_t>(p);
    s.hi = s.lo + static_cast<uintptr_t>(((rows - 1) * ld + width) * bytes);
    return s;
}
bool overlap(const Span &a, const Span &b) { return a.lo < b.hi && b.lo < a.hi; }
bool misaligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }
long long at_least_1(long long v) { return v > 1 ? v : 1; }

// Everything of a call, dense (E < 0) or by expert.
struct Call {
    int type, M, N, K, E;
    const int *offsets;
    const void *x, *w, *bias, *residual, *dy, *preact_in;
    void *preact, *y, *dx, *dw, *dbias;
    long long ldx, ldw, w_expert, ldr, ldz, ldy, lddy, lddx, lddw, dw_expert;
    int w_order, act;
    void *ws;
    size_t ws_bytes;
    cudaStream_t stream;
};
Call new_call(int type, int M, int N, int K, int E, const int *offsets) {
    Call c;
    memset(&c, 0, sizeof c);
    c.type = type;
    c.M = M;
    c.N = N;
    c.K = K;
    c.E = E;
    c.offsets = offsets;
    return c;
}
int experts(const Call &c) { return c.E < 0 ? 1 : c.E; }

int check_sizes(const Call &c) {
    if (c.type < LINEAR_F32 || c.type > LINEAR_F16 || c.act < LINEAR_ACT_NONE || c.act > LINEAR_ACT_GELU_TANH ||
        (c.w_order != 0 && c.w_order != 1))
        return SGEMM_ERR_INVALID_ARG;
    if (c.M < 0 || c.N < 0 || c.K < 0 || c.E < -1 || c.E > LINEAR_MAX_EXPERTS) return SGEMM_ERR_INVALID_DIM;
    // one coordinate past the last tile has to fit 32 bits
    if (c.M > INT_MAX - 1024 || c.N > INT_MAX - 1024 || c.K > INT_MAX - 1024) return SGEMM_ERR_INVALID_DIM;
    return SGEMM_OK;
}
bool weight_strides_bad(const Call &c, long long ld, long long expert) {
    const long long inner = c.w_order ? c.K : c.N, outer = c.w_order ? c.N : c.K;
    if (ld < at_least_1(inner)) return true;
    return c.E > 1 && expert < (outer - 1) * ld + inner;
}
Matrix weight_matrix(const Call &c) {
    Matrix m;
    m.base = c.w;
    m.inner = c.w_order ? c.K : c.N;
    m.outer = c.w_order ? c.N : c.K;
    m.planes = experts(c);
    m.ld = c.ldw;
    m.plane = c.E > 1 ? c.w_expert : m.outer * c.ldw;
    return m;
}
Span weight_span(const Call &c, const void *p, long long ld, long long expert) {
    const long long inner = c.w_order ? c.K : c.N, outer = c.w_order ? c.N : c.K;
    Span s = span(p, outer, inner, ld, lt::type_bytes(c.type));
    if (s.hi != 0 && c.E > 1) s.hi += static_cast<uintptr_t>((c.E - 1) * expert * lt::type_bytes(c.type));
    if (c.E == 0) s = Span();
    return s;
}
Matrix row_matrix(const void *p, int rows, int width, long long ld) {
    Matrix m;
    m.base = p;
    m.inner = width;
    m.outer = rows;
    m.ld = ld;
    m.plane = rows * ld;
    return m;
}

linear_few::Few few(const Call &c) {
    linear_few::Few p;
    memset(&p, 0, sizeof p);
    p.T = c.M, p.F = c.N, p.K = c.K, p.x = c.x, p.w = c.w, p.bias = c.bias, p.residual = c.residual;
    p.z = c.preact, p.out = c.y, p.ldx = c.ldx, p.ldw = c.ldw, p.ldr = c.ldr, p.ldz = c.ldz, p.ldo = c.ldy;
    p.order = c.w_order, p.act = c.act;
    return p;
}
bool few_tokens(const Call &c) { return c.E < 0 && c.K > 0 && linear_few::takes(c.type, few(c)); }

size_t forward_bytes(const Call &c) {
    if (check_sizes(c) != SGEMM_OK || c.M == 0 || c.N == 0 || c.K == 0 || c.E == 0 || few_tokens(c)) return 0;
    return operand_bytes(c.type, row_matrix(c.x, c.M, c.K, c.ldx)) + operand_bytes(c.type, weight_matrix(c));
}

int forward(const Call &c) {
    int st = check_sizes(c);
    if (st != SGEMM_OK) return st;
    const int b = lt::type_bytes(c.type);
    if (c.ldx < at_least_1(c.K) || weight_strides_bad(c, c.ldw, c.w_expert) || c.ldy < at_least_1(c.N) ||
        (c.residual != nullptr && c.ldr < at_least_1(c.N)) || (c.preact != nullptr && c.ldz < at_least_1(c.N)))
        return SGEMM_ERR_INVALID_LD;
    if (c.M == 0 || c.N == 0) return SGEMM_OK;
    if (c.y == nullptr || (c.E >= 0 && c.offsets == nullptr) ||
        (c.K > 0 && c.E != 0 && (c.x == nullptr || c.w == nullptr)))
        return SGEMM_ERR_NULL_PTR;
    const size_t need = forward_bytes(c);
    if (need > 0 && c.ws == nullptr) return SGEMM_ERR_NULL_PTR;
    if (misaligned(c.x, b) || misaligned(c.w, b) || misaligned(c.bias, b) || misaligned(c.residual, b) ||
        misaligned(c.preact, b) || misaligned(c.y, b) || misaligned(c.offsets, 4) || misaligned(c.ws, 256) ||
        c.ws_bytes < need)
        return SGEMM_ERR_INVALID_ARG;
    const Span sy = span(c.y, c.M, c.N, c.ldy, b), sz = span(c.preact, c.M, c.N, c.ldz, b),
               sr = span(c.residual, c.M, c.N, c.ldr, b), sws{reinterpret_cast<uintptr_t>(c.ws),
                                                              reinterpret_cast<uintptr_t>(c.ws) + need};
    const bool in_place = c.residual == c.y && c.ldr == c.ldy;
    const Span in[4] = {span(c.x, c.M, c.K, c.ldx, b), weight_span(c, c.w, c.ldw, c.w_expert),
                        span(c.bias, experts(c), c.N, c.N, b), span(c.offsets, 1, c.E + 1, 1, 4)};
    for (const Span &s : in)
        if (overlap(sy, s) || overlap(sz, s) || overlap(sws, s)) return SGEMM_ERR_ALIAS;
    if ((!in_place && overlap(sy, sr)) || overlap(sz, sr) || overlap(sws, sr) || overlap(sy, sz) || overlap(sws, sy) ||
        overlap(sws, sz))
        return SGEMM_ERR_ALIAS;
    Device d;
    st = set_up(&d);
    if (st != SGEMM_OK) return st;
    if (few_tokens(c)) {
        linear_few::Few p = few(c);
        p.sms = d.sms;
        if (linear_few::run(c.type, p, c.stream) == cudaSuccess) return SGEMM_OK;
        (void)cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    Operand P, Q;
    if (c.K > 0 && c.E != 0) {
        Copies copies(static_cast<char *>(c.ws));
        P = copies.operand(c.type, weight_matrix(c), c.w_order == 0);
        Q = copies.operand(c.type, row_matrix(c.x, c.M, c.K, c.ldx), false);
        st = copies.run(c.type, c.stream);
        if (st != SGEMM_OK) return st;
    }
    Product p;
    memset(&p, 0, sizeof p);
    p.T = c.M;
    p.F = c.N;
    p.K = c.E == 0 ? 0 : c.K;
    p.mode = c.E >= 0 ? ROWS_BY_EXPERT : DENSE;
    p.E = c.E > 0 ? c.E : 0;
    p.offsets = c.offsets;
    p.bias = c.bias;
    p.residual = c.residual;
    p.z = c.preact;
    p.out = c.y;
    p.ldr = c.ldr;
    p.ldz = c.ldz;
    p.ldo = c.ldy;
    p.act = c.act;
    return run_product(c.type, p, P, Q, d, c.stream);
}

struct Wanted {
    bool dx, dw, dbias;
};
// dz is a matrix of its own unless it is dy and the tensor copies can read that.
bool dz_is_dy(const Call &c) {
    return c.act == LINEAR_ACT_NONE && direct(c.type, row_matrix(c.dy, c.M, c.N, c.lddy));
}
struct BackwardBytes {
    size_t dz, x, w, sums, total;
};
BackwardBytes backward_bytes(const Call &c, const Wanted &want) {
    BackwardBytes r;
    memset(&r, 0, sizeof r);
    if (check_sizes(c) != SGEMM_OK || c.M == 0 || c.N == 0 || c.E == 0) return r;
    if ((want.dx || want.dw) && c.K > 0) {
        if (!dz_is_dy(c)) r.dz = up256(c.M * up8(c.N) * 2 * (c.type == LINEAR_F32 ? 3 : 1));
        if (want.dw) r.x = operand_bytes(c.type, row_matrix(c.x, c.M, c.K, c.ldx));
        if (want.dx) r.w = operand_bytes(c.type, weight_matrix(c));
    }
    if (want.dbias) r.sums = up256(linear_prep::sums_bytes(c.M, c.N, experts(c)));
    r.total = r.dz + r.x + r.w + r.sums;
    return r;
}

int backward(const Call &c) {
    int st = check_sizes(c);
    if (st != SGEMM_OK) return st;
    const int b = lt::type_bytes(c.type);
    const Wanted want{c.dx != nullptr, c.dw != nullptr, c.dbias != nullptr};
    if (c.lddy < at_least_1(c.N) || (want.dw && c.ldx < at_least_1(c.K)) ||
        (want.dx && (weight_strides_bad(c, c.ldw, c.w_expert) || c.lddx < at_least_1(c.K))) ||
        (want.dw && weight_strides_bad(c, c.lddw, c.dw_expert)) ||
        (c.act != LINEAR_ACT_NONE && c.ldz < at_least_1(c.N)))
        return SGEMM_ERR_INVALID_LD;
    if ((c.preact_in != nullptr) != (c.act != LINEAR_ACT_NONE) && c.M > 0 && c.N > 0) return SGEMM_ERR_INVALID_ARG;
    if (!want.dx && !want.dw && !want.dbias) return SGEMM_OK;
    if (c.M > 0 && c.N > 0) {
        if (c.dy == nullptr || (c.E >= 0 && c.offsets == nullptr) ||
            (c.K > 0 && c.E != 0 && ((want.dw && c.x == nullptr) || (want.dx && c.w == nullptr))))
            return SGEMM_ERR_NULL_PTR;
    }
    const BackwardBytes need = backward_bytes(c, want);
    if (need.total > 0 && c.ws == nullptr) return SGEMM_ERR_NULL_PTR;
    if (misaligned(c.dy, b) || misaligned(c.x, b) || misaligned(c.w, b) || misaligned(c.preact_in, b) ||
        misaligned(c.dx, b) || misaligned(c.dw, b) || misaligned(c.dbias, b) || misaligned(c.offsets, 4) ||
        misaligned(c.ws, 256) || c.ws_bytes < need.total)
        return SGEMM_ERR_INVALID_ARG;
    const Span in[5] = {span(c.dy, c.M, c.N, c.lddy, b),
                        want.dw ? span(c.x, c.M, c.K, c.ldx, b) : Span(),
                        want.dx ? weight_span(c, c.w, c.ldw, c.w_expert) : Span(),
                        span(c.preact_in, c.M, c.N, c.ldz, b), span(c.offsets, 1, c.E + 1, 1, 4)};
    const Span out[4] = {span(c.dx, c.M, c.K, c.lddx, b), weight_span(c, c.dw, c.lddw, c.dw_expert),
                         span(c.dbias, experts(c), c.N, c.N, b),
                         {reinterpret_cast<uintptr_t>(c.ws), reinterpret_cast<uintptr_t>(c.ws) + need.total}};
    for (int i = 0; i < 4; ++i) {
        for (const Span &s : in)
            if (overlap(out[i], s)) return SGEMM_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return SGEMM_ERR_ALIAS;
    }
    Device d;
    st = set_up(&d);
    if (st != SGEMM_OK) return st;
    char *ws = static_cast<char *>(c.ws);
    const bool products = (want.dx || want.dw) && c.K > 0;
    const bool empty = c.M == 0 || c.N == 0 || c.E == 0;
    Product p;
    memset(&p, 0, sizeof p);
    // the weight and x, where they need a copy (the weight, then x), dz and the column sums
    Operand P_dx, X;
    if (!empty && products) {
        Copies copies(ws + need.dz + need.sums);
        if (want.dx) P_dx = copies.operand(c.type, weight_matrix(c), c.w_order == 1);
        if (want.dw) X = copies.operand(c.type, row_matrix(c.x, c.M, c.K, c.ldx), true);
        st = copies.run(c.type, c.stream);
        if (st != SGEMM_OK) return st;
    }
    Operand dz;  // M rows of N
    dz.inner = c.N;
    dz.outer = c.M;
    if (!empty) {
        const bool make = products && !dz_is_dy(c);
        if (dz_is_dy(c)) {
            dz.base = c.dy;
            dz.ld = c.lddy;
        } else {
            dz.base = ws;
            dz.ld = up8(c.N);
            dz.plane = c.M * dz.ld;
            if (c.type == LINEAR_F32) dz.planes = 3;
        }
        float *sums = want.dbias ? reinterpret_cast<float *>(ws + need.dz) : nullptr;
        cudaError_t err = linear_prep::activation_gradient(c.type, c.act, c.M, c.N, c.E, c.offsets, c.dy, c.lddy,
                                                           c.preact_in, c.ldz, make ? ws : nullptr, dz.ld, sums, c.stream);
        if (want.dbias && products) {  // a warp of the first product adds them up
            p.sums = sums;
            p.dbias = c.dbias;
            p.sums_M = c.M;
            p.sums_N = c.N;
            p.sums_E = c.E;
        } else if (want.dbias && err == cudaSuccess) {
            err = linear_prep::column_sums(c.type, c.M, c.N, c.E, c.offsets, sums, c.dbias, c.stream);
        }
        if (err != cudaSuccess) {
            (void)cudaGetLastError();
            return SGEMM_ERR_LAUNCH;
        }
    } else if (want.dbias && c.N > 0) {
        if (cudaMemsetAsync(c.dbias, 0, static_cast<size_t>(experts(c)) * c.N * b, c.stream) != cudaSuccess) {
            (void)cudaGetLastError();
            return SGEMM_ERR_LAUNCH;
        }
    }
    if (!products) return SGEMM_OK;
    p.offsets = c.offsets;
    p.E = c.E > 0 ? c.E : 0;
    if (want.dx && c.M > 0) {
        Operand Q = dz;
        Q.mn = false;
        p.T = c.M;
        p.F = c.K;
        p.K = empty ? 0 : c.N;
        p.mode = c.E >= 0 && !empty ? ROWS_BY_EXPERT : DENSE;
        p.out = c.dx;
        p.ldo = c.lddx;
        const bool two = !empty && want.dw;
        p.order = two ? ORDER_FIRST : ORDER_ALONE;
        st = run_product(c.type, p, P_dx, Q, d, c.stream);
        if (st != SGEMM_OK) return st;
        p.dbias = nullptr;
        p.order = two ? ORDER_BESIDE : ORDER_ALONE;
    }
    if (want.dw && c.N > 0 && c.E != 0) {
        Operand Z = dz;
        Z.mn = true;
        // rows of dw in memory: K of N (order 0) or N of K (order 1)
        p.T = c.w_order ? c.N : c.K;
        p.F = c.w_order ? c.K : c.N;
        p.K = empty ? 0 : c.M;
        p.mode = c.E >= 0 ? K_BY_EXPERT : DENSE;  // without rows every expert's is zero
        p.out = c.dw;
        p.ldo = c.lddw;
        p.out_expert = c.E > 1 ? c.dw_expert : 0;
        st = run_product(c.type, p, c.w_order ? X : Z, c.w_order ? Z : X, d, c.stream);
        if (st != SGEMM_OK) return st;
    }
    return SGEMM_OK;
}

}  // namespace

extern "C" int linear_forward(int type, int M, int N, int K, const void *x, int64_t ldx, const void *w, int64_t ldw,
                              int w_order, const void *bias, const void *residual, int64_t ldr, int activation,
                              void *preact, int64_t ldz, void *y, int64_t ldy, void *workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
    Call c = new_call(type, M, N, K, -1, nullptr);
    c.x = x, c.ldx = ldx, c.w = w, c.ldw = ldw, c.w_order = w_order, c.bias = bias, c.residual = residual, c.ldr = ldr;
    c.act = activation, c.preact = preact, c.ldz = ldz, c.y = y, c.ldy = ldy;
    c.ws = workspace, c.ws_bytes = workspace_bytes, c.stream = stream;
    return forward(c);
}

extern "C" size_t linear_forward_workspace_size(int type, int M, int N, int K, const void *x, int64_t ldx,
                                                const void *w, int64_t ldw, int w_order) {
    Call c = new_call(type, M, N, K, -1, nullptr);
    c.x = x, c.ldx = ldx, c.w = w, c.ldw = ldw, c.w_order = w_order;
    return forward_bytes(c);
}

extern "C" int expert_linear_forward(int type, int R, int N, int K, int E, const int *offsets, const void *x,
                                     int64_t ldx, const void *w, int64_t ldw, int64_t w_expert, int w_order,
                                     const void *bias, const void *residual, int64_t ldr, int activation,
                                     void *preact, int64_t ldz, void *y, int64_t ldy, void *workspace,
                                     size_t workspace_bytes, cudaStream_t stream) {
    if (E < 0) return SGEMM_ERR_INVALID_DIM;
    Call c = new_call(type, R, N, K, E, offsets);
    c.x = x, c.ldx = ldx, c.w = w, c.ldw = ldw, c.w_expert = w_expert, c.w_order = w_order, c.bias = bias;
    c.residual = residual, c.ldr = ldr, c.act = activation, c.preact = preact, c.ldz = ldz, c.y = y, c.ldy = ldy;
    c.ws = workspace, c.ws_bytes = workspace_bytes, c.stream = stream;
    return forward(c);
}

extern "C" size_t expert_linear_forward_workspace_size(int type, int R, int N, int K, int E, const void *x,
                                                       int64_t ldx, const void *w, int64_t ldw, int64_t w_expert,
                                                       int w_order) {
    if (E < 0) return 0;
    Call c = new_call(type, R, N, K, E, nullptr);
    c.x = x, c.ldx = ldx, c.w = w, c.ldw = ldw, c.w_expert = w_expert, c.w_order = w_order;
    return forward_bytes(c);
}

extern "C" int linear_backward(int type, int M, int N, int K, const void *dy, int64_t lddy, const void *x,
                               int64_t ldx, const void *w, int64_t ldw, int w_order, const void *preact, int64_t ldz,
                               int activation, void *dx, int64_t lddx, void *dw, int64_t lddw, void *dbias,
                               void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    Call c = new_call(type, M, N, K, -1, nullptr);
    c.dy = dy, c.lddy = lddy, c.x = x, c.ldx = ldx, c.w = w, c.ldw = ldw, c.w_order = w_order;
    c.preact_in = preact, c.ldz = ldz, c.act = activation, c.dx = dx, c.lddx = lddx, c.dw = dw, c.lddw = lddw;
    c.dbias = dbias, c.ws = workspace, c.ws_bytes = workspace_bytes, c.stream = stream;
    return backward(c);
}

extern "C" size_t linear_backward_workspace_size(int type, int M, int N, int K, const void *dy, int64_t lddy,
                                                 const void *x, int64_t ldx, const void *w, int64_t ldw, int w_order,
                                                 int activation, int want_dx, int want_dw, int want_dbias) {
    Call c = new_call(type, M, N, K, -1, nullptr);
    c.dy = dy, c.lddy = lddy, c.x = x, c.ldx = ldx, c.w = w, c.ldw = ldw, c.w_order = w_order, c.act = activation;
    return backward_bytes(c, Wanted{want_dx != 0, want_dw != 0, want_dbias != 0}).total;
}

extern "C" int expert_linear_backward(int type, int R, int N, int K, int E, const int *offsets, const void *dy,
                                      int64_t lddy, const void *x, int64_t ldx, const void *w, int64_t ldw,
                                      int64_t w_expert, int w_order, const void *preact, int64_t ldz, int activation,
                                      void *dx, int64_t lddx, void *dw, int64_t lddw, int64_t dw_expert, void *dbias,
                                      void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (E < 0) return SGEMM_ERR_INVALID_DIM;
    Call c = new_call(type, R, N, K, E, offsets);
    c.dy = dy, c.lddy = lddy, c.x = x, c.ldx = ldx, c.w = w, c.ldw = ldw, c.w_expert = w_expert, c.w_order = w_order;
    c.preact_in = preact, c.ldz = ldz, c.act = activation, c.dx = dx, c.lddx = lddx, c.dw = dw, c.lddw = lddw;
    c.dw_expert = dw_expert, c.dbias = dbias, c.ws = workspace, c.ws_bytes = workspace_bytes, c.stream = stream;
    return backward(c);
}

extern "C" size_t expert_linear_backward_workspace_size(int type, int R, int N, int K, int E, const void *dy,
                                                        int64_t lddy, const void *x, int64_t ldx, const void *w,
                                                        int64_t ldw, int64_t w_expert, int w_order, int activation,
                                                        int want_dx, int want_dw, int want_dbias) {
    if (E < 0) return 0;
    Call c = new_call(type, R, N, K, E, nullptr);
    c.dy = dy, c.lddy = lddy, c.x = x, c.ldx = ldx, c.w = w, c.ldw = ldw, c.w_expert = w_expert, c.w_order = w_order;
    c.act = activation;
    return backward_bytes(c, Wanted{want_dx != 0, want_dw != 0, want_dbias != 0}).total;
}

extern "C" int linear_timeouts(unsigned *count) {
    if (count == nullptr) return SGEMM_ERR_NULL_PTR;
    if (cudaMemcpyFromSymbol(count, g_linear_timeout, sizeof(unsigned)) != cudaSuccess) {
        (void)cudaGetLastError();
        return SGEMM_ERR_DEVICE;
    }
    return SGEMM_OK;
}
