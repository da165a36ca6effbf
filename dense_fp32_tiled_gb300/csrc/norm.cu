// norm.cu -- layer norm and its gradient (C ABI: include/norm.h).  Bound by
// HBM: the forward pass reads and writes each value once, the gradient reads
// two and writes one.
//
// A row is held in the registers of a warp, or a block, while its sums go round:
// of each warp's 32 * PPT packs of V values, lane k has k, k + 32, ...  (Steps of a
// constant size: one address serves all of a thread's accesses to a row.)  The mean is rounded; the
// differences to it are summed again, which gives what the rounding left, and
// squared for the variance, which so has no cancellation.
//
// At HBM's rate an SM has 0.9 clocks for a value of the forward pass and 1.4 for
// one of the gradient, so instructions count: arithmetic on pairs, no
// division in a row, and registers no larger than leave the SM its warps.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "linear_types.cuh"
#include "norm.h"
#include "nvtx_range.cuh"
#include "rows.cuh"
#include "tensor_core.cuh"

namespace {

using namespace rows;

constexpr int MOST_THREADS = 512;       // of a row held in registers
constexpr int MANY_THREADS = 768;       // of a block of several rows, if they hold 16 values each
constexpr int MOST_WARPS = 24;

// The sums of N values over the threads of a row (blockDim.x of them), the same
// in each: across the warp, then over the warps, in a fixed order.  The lanes
// share the values out first (of three, lanes 0-7 add up the first, 8-15 the
// second, 16-23 the third), which takes 6 exchanges for 15.  `part` has two sets,
// used in turn (`turn`), so that one barrier a sum is enough.  SEVERAL: the
// block's rows (threadIdx.y) have barriers of their own.  (A barrier whose number
// is not a constant takes all 16 of a block, and an SM has them for four blocks.)
__device__ __forceinline__ float across(float v, int k) { return v + __shfl_xor_sync(0xffffffffu, v, k); }
template <bool SEVERAL, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*part)[MOST_WARPS][4], int &turn) {
    constexpr int SHARE = N == 1 ? 32 : N == 2 ? 16 : 8;  // lanes of a value
    const int lane = threadIdx.x & 31;
    float t;
    if constexpr (N == 1) {
        t = across(v[0], 16);
        t = across(t, 8);
    } else {
        const bool upper = (lane & 16) != 0;
        if constexpr (N == 2) {
            t = (upper ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, upper ? v[0] : v[1], 16);
            t = across(t, 8);
        } else {
            const float a = (upper ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, upper ? v[0] : v[2], 16);
            const float b = across(v[1], 16);
            const bool odd = (lane & 8) != 0;
            t = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
        }
    }
    t = across(t, 4);
    t = across(t, 2);
    t = across(t, 1);
    if (blockDim.x > 32) {
        const int warps = blockDim.x >> 5, first = threadIdx.y * warps;
        if ((lane & (SHARE - 1)) == 0) part[turn][first + (threadIdx.x >> 5)][lane / SHARE] = t;
        if constexpr (SEVERAL)
            asm volatile("bar.sync %0, %1;\n" ::"r"(1 + threadIdx.y), "r"(blockDim.x) : "memory");
        else
            asm volatile("bar.sync 0;\n" ::: "memory");  // reached from either of a kernel's two loops
        t = 0.0f;
        for (int w = lane & 7; w < warps; w += 8) t += part[turn][first + w][N == 1 ? 0 : lane / SHARE];
        t = across(t, 4);
        t = across(t, 2);
        t = across(t, 1);
        turn ^= 1;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = N == 1 ? t : __shfl_sync(0xffffffffu, t, i * SHARE);
}

// The packs of a thread's next row, on their way while it works on this one: in
// slots of shared memory that only this thread reads, so no barrier is needed
// (2-byte packs, which no asynchronous copy moves: in registers).  COUNT matrices
// of PPT packs each; two rows' room.  (Two rows ahead took longer while weights came from
// the L1 that their room takes: 16384 x 4096 bf16 62 us for 47.)
template <typename T, int V, int PPT, int COUNT, int THREADS>
struct Ahead {
    using P = Pack<T, V>;
    static constexpr bool ASYNC = P::BYTES >= 4;
    static constexpr int SLOT = ASYNC ? P::BYTES : 0;
    static constexpr int APART = THREADS * SLOT, ROOM = COUNT * PPT * APART;
    uint32_t at;    // this thread's first slot of the row at work
    int other;      // how far from it the next row's is
    P held[ASYNC ? 1 : COUNT * PPT], next[ASYNC ? 1 : COUNT * PPT];
    __device__ __forceinline__ explicit Ahead(void *room) {
        at = tc::smem_u32(room) + (threadIdx.y * blockDim.x + threadIdx.x) * SLOT + ROOM;
        other = -ROOM;
    }
    __device__ __forceinline__ void ask(int m, int i, bool in, const T *src) {
        if constexpr (ASYNC) {
            const uint32_t to = at + other + (m * PPT + i) * APART;
            if (in) {
                if constexpr (P::BYTES == 16)
                    tc::cp_async16(to, src);
                else
                    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(to), "l"(src), "n"(P::BYTES < 4 ? 4 : P::BYTES) : "memory");
            }
        } else {
            next[m * PPT + i] = load_if<T, V>(in, src);
        }
    }
    // A row has been asked for whole.
    __device__ __forceinline__ void asked() {
        if constexpr (ASYNC) tc::cp_async_commit();
    }
    // The row at work is over, the one asked for is next.
    __device__ __forceinline__ void turn() {
        if constexpr (ASYNC) {
            at += other;
            other = -other;
            tc::cp_async_wait<0>();
        } else {
#pragma unroll
            for (int i = 0; i < COUNT * PPT; ++i) held[i] = next[i];
        }
    }
    __device__ __forceinline__ P get(int m, int i) const {
        if constexpr (ASYNC) {
            const uint32_t from = at + (m * PPT + i) * APART;
            P p;
            if constexpr (P::BYTES == 16)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(p.raw.x), "=r"(p.raw.y), "=r"(p.raw.z), "=r"(p.raw.w) : "r"(from));
            else if constexpr (P::BYTES == 8)
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(p.raw.x), "=r"(p.raw.y) : "r"(from));
            else if constexpr (P::BYTES == 4)
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(p.raw) : "r"(from));
            return p;
        } else {
            return held[m * PPT + i];
        }
    }
};

struct Forward {
    const void *x, *weight, *bias;
    void *y;
    float *stats;
    long long ldx, ldy;
    int M, N, packs;
    float eps, inverse;  // 1 / N
};

// What the passes over a row's packs do.
template <typename T, int V>
struct Row {
    using L = Lanes<V>;
    using Num = typename L::Num;
    using P = Pack<T, V>;
    static __device__ __forceinline__ void add_up(const P &x, Num (&f)[L::N], Num &s) {
        get<T, V>(x, f);
#pragma unroll
        for (int k = 0; k < L::N; ++k) s = add(s, f[k]);
    }
    // the differences to the mean, their sum and that of their squares
    static __device__ __forceinline__ void spread(Num (&f)[L::N], Num minus_mean, Num &s, Num &q) {
#pragma unroll
        for (int k = 0; k < L::N; ++k) {
            f[k] = add(f[k], minus_mean);
            s = add(s, f[k]);
            q = fma_of(f[k], f[k], q);
        }
    }
    // (d rstd - rest rstd) w + b
    static __device__ __forceinline__ void finish(Num (&f)[L::N], const P &w, const P &b, Num rstd, Num minus_rest, T *y) {
        Num fw[L::N], fb[L::N];
        get<T, V>(w, fw);
        get<T, V>(b, fb);
#pragma unroll
        for (int k = 0; k < L::N; ++k) f[k] = fma_of(fma_of(f[k], rstd, minus_rest), fw[k], fb[k]);
        store<T, V>(y, pack_of<T, V>(f));
    }
    // sums of g w, of g w d and of d
    static __device__ __forceinline__ void means(const P &x, const P &g, const P &w, Num minus_mean, Num &sg, Num &sgd, Num &sd) {
        Num fx[L::N], fg[L::N], fw[L::N];
        get<T, V>(x, fx);
        get<T, V>(g, fg);
        get<T, V>(w, fw);
#pragma unroll
        for (int k = 0; k < L::N; ++k) {
            const Num d = add(fx[k], minus_mean), gw = mul(fg[k], fw[k]);
            sg = add(sg, gw);
            sgd = fma_of(gw, d, sgd);
            sd = add(sd, d);
        }
    }
    // dx = rstd g w + (a d + b), and the columns' sums of g h and g
    static __device__ __forceinline__ P gradient(const P &x, const P &g, const P &w, Num minus_mean, Num rstd, Num minus_rest, Num a,
                                                 Num b, Num (&dw)[L::N], Num (&db)[L::N]) {
        Num fx[L::N], fg[L::N], fw[L::N];
        get<T, V>(x, fx);
        get<T, V>(g, fg);
        get<T, V>(w, fw);
#pragma unroll
        for (int k = 0; k < L::N; ++k) {
            const Num d = add(fx[k], minus_mean);
            dw[k] = fma_of(fg[k], fma_of(d, rstd, minus_rest), dw[k]);
            db[k] = add(db[k], fg[k]);
            fx[k] = fma_of(mul(fg[k], fw[k]), rstd, fma_of(d, a, b));
        }
        return pack_of<T, V>(fx);
    }
};

struct Spread {
    float rest, rstd;
};
__device__ __forceinline__ Spread spread_of(const Forward &c, const float (&q)[2]) {
    const float rest = q[0] * c.inverse, var = fmaf(-rest, rest, q[1] * c.inverse);
    return {rest, 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + c.eps)};  // a NaN stays one
}

// The loop over the rows is there twice: for warps whose share is whole, with a
// weight and a bias (the gradient: a weight and dx), so that nothing is asked in a
// row, and for the others.
struct Yes {
    static constexpr bool value = true;
};
struct No {
    static constexpr bool value = false;
};

// PPT packs a thread.  A block takes every blocks-th row (of each of its
// threadIdx.y) and asks for its next row before it sums up this one.
// SEVERAL: one block an SM, of as many rows as it has threads for, with weight and bias
// in shared memory.  They could come from L1 for each row, in blocks of a row, of which
// an SM has several; but narrow asynchronous copies go through L1 and drive them out, and
// blocks' rooms are less of an SM's the wider the rows (us; there, here: 16384 x 4096
// bf16 46.4, 43.4; 8192 x 5120 f32 88, 60; 8188 x 4098 f32 128, 57; 60000 x 1001 bf16
// 141, 76).  Rows of a warp and rows of which a block has one are there all the same
// (60000 x 128 f32 18.4 us, here 20.5).
template <typename T, int V, int PPT, int THREADS, bool SEVERAL>
__global__ void __launch_bounds__(THREADS, SEVERAL ? 1 : 1024 / THREADS) forward_kernel(const __grid_constant__ Forward c) {
    using R = Row<T, V>;
    using Num = typename R::Num;
    using P = Pack<T, V>;
    using A = Ahead<T, V, PPT, 1, THREADS>;
    __shared__ __align__(16) float part[2][MOST_WARPS][4];
    extern __shared__ __align__(16) uint8_t room[];
    const long long step = static_cast<long long>(gridDim.x) * blockDim.y;
    long long r = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    const T *wp = static_cast<const T *>(c.weight), *bp = static_cast<const T *>(c.bias);
    A ahead(room);
    const int p0 = (threadIdx.x & ~31) * PPT + (threadIdx.x & 31);
    P *const ws = reinterpret_cast<P *>(room + 2 * A::ROOM), *const bs = ws + c.packs;
    tc::grid_trigger();
    tc::grid_wait();
    auto rows = [&](auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        auto mine = [&](int i) { return WHOLE || p0 + 32 * i < c.packs; };
        auto ask = [&](long long row) {
            if (row < c.M) {
                const T *x = static_cast<const T *>(c.x) + row * c.ldx + p0 * V;
#pragma unroll
                for (int i = 0; i < PPT; ++i) ahead.ask(0, i, mine(i), x + 32 * i * V);
            }
            ahead.asked();
        };
        ask(r);
        if constexpr (SEVERAL) {
            for (int p = threadIdx.y * blockDim.x + threadIdx.x; p < c.packs; p += blockDim.x * blockDim.y) {
                ws[p] = load_or_ones<T, V>(wp != nullptr, wp + static_cast<long long>(p) * V);
                bs[p] = load_if<T, V>(bp != nullptr, bp + static_cast<long long>(p) * V);
            }
            asm volatile("bar.sync 0;\n" ::: "memory");
        }
        int turn = 0;
        for (; r < c.M; r += step) {
            ahead.turn();
            Num f[PPT][R::L::N], sum = all<Num>(0.0f), square = sum;
#pragma unroll
            for (int i = 0; i < PPT; ++i)
                if (mine(i)) R::add_up(ahead.get(0, i), f[i], sum);
            ask(r + step);
            float s[1] = {sum_of(sum)};
            row_sum<SEVERAL>(s, part, turn);
            const float mean = s[0] * c.inverse;
            const Num minus_mean = all<Num>(-mean);
            sum = all<Num>(0.0f);
#pragma unroll
            for (int i = 0; i < PPT; ++i)
                if (mine(i)) R::spread(f[i], minus_mean, sum, square);
            float q[2] = {sum_of(sum), sum_of(square)};
            row_sum<SEVERAL>(q, part, turn);
            const Spread sp = spread_of(c, q);
            if (c.stats != nullptr && threadIdx.x == 0) {
                c.stats[2 * r] = mean + sp.rest;
                c.stats[2 * r + 1] = sp.rstd;
            }
            const Num rstd = all<Num>(sp.rstd), minus_rest = all<Num>(-sp.rest * sp.rstd);
            T *y = static_cast<T *>(c.y) + r * c.ldy;
#pragma unroll
            for (int i = 0; i < PPT; ++i) {
                const int p = p0 + 32 * i;
                if (!mine(i)) continue;
                if constexpr (SEVERAL)
                    R::finish(f[i], ws[p], bs[p], rstd, minus_rest, y + p * V);
                else
                    R::finish(f[i], load_or_ones<T, V>(WHOLE || wp != nullptr, wp + p * V), load_if<T, V>(WHOLE || bp != nullptr, bp + p * V),
                              rstd, minus_rest, y + p * V);
            }
        }
    };
    if ((threadIdx.x & ~31) * PPT + 32 * PPT <= c.packs && (SEVERAL || (wp != nullptr && bp != nullptr)))
        rows(Yes());
    else
        rows(No());
}

// Rows that no block's registers hold: read three times, the later ones from L2.
template <typename T, int V>
__global__ void __launch_bounds__(MOST_THREADS) forward_wide_kernel(const __grid_constant__ Forward c) {
    using R = Row<T, V>;
    using Num = typename R::Num;
    __shared__ __align__(16) float part[2][MOST_WARPS][4];
    const long long r = blockIdx.x;
    tc::grid_trigger();
    tc::grid_wait();
    const T *row = static_cast<const T *>(c.x) + r * c.ldx;
    const T *wp = static_cast<const T *>(c.weight), *bp = static_cast<const T *>(c.bias);
    int turn = 0;
    Num sum = all<Num>(0.0f), square = sum;
#pragma unroll 4
    for (int p = threadIdx.x; p < c.packs; p += blockDim.x) {
        Num f[R::L::N];
        R::add_up(load<T, V>(row + static_cast<long long>(p) * V), f, sum);
    }
    float s[1] = {sum_of(sum)};
    row_sum<false>(s, part, turn);
    const float mean = s[0] * c.inverse;
    const Num minus_mean = all<Num>(-mean);
    sum = all<Num>(0.0f);
#pragma unroll 4
    for (int p = threadIdx.x; p < c.packs; p += blockDim.x) {
        Num f[R::L::N];
        get<T, V>(load<T, V>(row + static_cast<long long>(p) * V), f);
        R::spread(f, minus_mean, sum, square);
    }
    float q[2] = {sum_of(sum), sum_of(square)};
    row_sum<false>(q, part, turn);
    const Spread sp = spread_of(c, q);
    if (c.stats != nullptr && threadIdx.x == 0) {
        c.stats[2 * r] = mean + sp.rest;
        c.stats[2 * r + 1] = sp.rstd;
    }
    const Num rstd = all<Num>(sp.rstd), minus_rest = all<Num>(-sp.rest * sp.rstd);
    T *y = static_cast<T *>(c.y) + r * c.ldy;
#pragma unroll 4
    for (int p = threadIdx.x; p < c.packs; p += blockDim.x) {
        const long long at = static_cast<long long>(p) * V;
        Num f[R::L::N];
        get<T, V>(load<T, V>(row + at), f);
#pragma unroll
        for (int k = 0; k < R::L::N; ++k) f[k] = add(f[k], minus_mean);
        R::finish(f, load_or_ones<T, V>(wp != nullptr, wp + at), load_if<T, V>(bp != nullptr, bp + at), rstd, minus_rest, y + at);
    }
}

// ---- gradient -----------------------------------------------------------------------
struct Backward {
    const void *dy, *x, *weight;
    const float *stats;
    void *dx, *dweight, *dbias;
    float *sums;  // blocks x 2 x N: each block's part of dweight and dbias
    float *rest;  // wide rows: what rounding left of their mean
    long long lddy, ldx, lddx;
    int M, N, packs, blocks;
    float inverse;  // 1 / N
};

// Of a row's sums of g, of g d and of d (d = x - mean): with rest, the mean of d,
// h = (d - rest) rstd, and dx = rstd (g - mean g - h mean(g h)) = rstd g + a d + b.
struct RowMeans {
    float rest, a, b;
};
__device__ __forceinline__ RowMeans row_means(const float (&q)[3], float inverse, float rstd) {
    const float rest = q[2] * inverse, g = q[0] * inverse;
    const float gh = fmaf(q[1], inverse, -rest * g) * rstd;
    const float a = -rstd * rstd * gh;
    return {rest, a, fmaf(-rest, a, -rstd * g)};
}

// A grid of `blocks` blocks, one an SM, takes the rows in turn, one each of their
// threadIdx.y at a time; a thread keeps the sums of its columns in registers, and
// the block's are joined in shared memory at the end.  Each row's packs are read
// from their slots twice, before and after its means are known.  Weights are in shared
// memory (16384 x 4096 bf16 69 us, from L1 for each row 77; 16380 x 4097 154, held in
// registers 174); FP32 ones by 4 bytes stay in registers, and those of wide FP32 rows, which
// leave no room there, and of 16-bit rows of a pack a lane come from L1.
template <typename T, int V, int PPT, int THREADS, bool SHARED_WEIGHT>
__global__ void __launch_bounds__(THREADS) backward_kernel(const __grid_constant__ Backward c) {
    using R = Row<T, V>;
    using Num = typename R::Num;
    constexpr int LN = R::L::N;
    __shared__ __align__(16) float part[2][MOST_WARPS][4];
    extern __shared__ __align__(16) uint8_t room[];
    Num dw[PPT][LN], db[PPT][LN];
#pragma unroll
    for (int i = 0; i < PPT; ++i)
#pragma unroll
        for (int k = 0; k < LN; ++k) dw[i][k] = db[i][k] = all<Num>(0.0f);
    const T *wp = static_cast<const T *>(c.weight);
    const long long step = static_cast<long long>(c.blocks) * blockDim.y;
    long long r = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    Ahead<T, V, PPT, 2, THREADS> ahead(room);
    const int p0 = (threadIdx.x & ~31) * PPT + (threadIdx.x & 31);
    constexpr bool HOLD = std::is_same<T, float>::value && V == 1;
    Pack<T, V> *const ws = reinterpret_cast<Pack<T, V> *>(room + 2 * decltype(ahead)::ROOM);
    float next_mean = 0.0f, next_rstd = 0.0f;
    tc::grid_trigger();
    tc::grid_wait();
    auto rows = [&](auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        auto mine = [&](int i) { return WHOLE || p0 + 32 * i < c.packs; };
        auto ask = [&](long long row) {
            if (row < c.M) {
                const T *xr = static_cast<const T *>(c.x) + row * c.ldx + p0 * V, *gr = static_cast<const T *>(c.dy) + row * c.lddy + p0 * V;
#pragma unroll
                for (int i = 0; i < PPT; ++i) {
                    ahead.ask(0, i, mine(i), xr + 32 * i * V);
                    ahead.ask(1, i, mine(i), gr + 32 * i * V);
                }
                next_mean = c.stats[2 * row];
                next_rstd = c.stats[2 * row + 1];
            }
            ahead.asked();
        };
        ask(r);
        Pack<T, V> held[HOLD ? PPT : 1];
        if constexpr (SHARED_WEIGHT) {
            for (int p = threadIdx.y * blockDim.x + threadIdx.x; p < c.packs; p += blockDim.x * blockDim.y)
                ws[p] = load_or_ones<T, V>(wp != nullptr, wp + static_cast<long long>(p) * V);
            asm volatile("bar.sync 0;\n" ::: "memory");
        }
        auto fetch_weight = [&](int i) { return load_or_ones<T, V>(WHOLE || (mine(i) && wp != nullptr), wp + (p0 + 32 * i) * V); };
        if constexpr (HOLD) {
#pragma unroll
            for (int i = 0; i < PPT; ++i) held[i] = fetch_weight(i);
        }
        auto weight = [&](int i) {
            if constexpr (HOLD)
                return held[i];
            else if constexpr (SHARED_WEIGHT)
                return ws[p0 + 32 * i];
            else
                return fetch_weight(i);
        };
        int turn = 0;
        for (; r < c.M; r += step) {
            ahead.turn();
            const float rstd = next_rstd;
            const Num minus_mean = all<Num>(-next_mean);
            ask(r + step);
            Num sg = all<Num>(0.0f), sgd = sg, sd = sg;
#pragma unroll
            for (int i = 0; i < PPT; ++i)
                if (mine(i)) R::means(ahead.get(0, i), ahead.get(1, i), weight(i), minus_mean, sg, sgd, sd);
            float q[3] = {sum_of(sg), sum_of(sgd), sum_of(sd)};
            row_sum<true>(q, part, turn);
            const RowMeans m = row_means(q, c.inverse, rstd);
            const Num n_rstd = all<Num>(rstd), minus_rest = all<Num>(-m.rest * rstd), a = all<Num>(m.a), b = all<Num>(m.b);
            T *dx = static_cast<T *>(c.dx) + r * c.lddx;
#pragma unroll
            for (int i = 0; i < PPT; ++i)
                if (mine(i)) {
                    const Pack<T, V> o = R::gradient(ahead.get(0, i), ahead.get(1, i), weight(i), minus_mean, n_rstd, minus_rest, a, b, dw[i], db[i]);
                    if (WHOLE || c.dx != nullptr) store<T, V>(dx + (p0 + 32 * i) * V, o);
                }
        }
    };
    if ((threadIdx.x & ~31) * PPT + 32 * PPT <= c.packs && wp != nullptr && c.dx != nullptr)
        rows(Yes());
    else
        rows(No());
    if (c.sums == nullptr) return;
    // the rows' sums, in their order: V values of a thread lie together, so no two threads share any
    float *joined = reinterpret_cast<float *>(room);
    for (int y = 0; y < static_cast<int>(blockDim.y); ++y) {
        __syncthreads();
        if (y != static_cast<int>(threadIdx.y)) continue;
#pragma unroll
        for (int i = 0; i < PPT; ++i) {
            const int p = p0 + 32 * i;
            if (p < c.packs)
#pragma unroll
                for (int k = 0; k < LN; ++k)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        Num *at = reinterpret_cast<Num *>(joined + s * c.N + p * V) + k;
                        const Num v = s == 0 ? dw[i][k] : db[i][k];
                        *at = y == 0 ? v : add(*at, v);
                    }
        }
    }
    __syncthreads();
    float *to = c.sums + static_cast<long long>(blockIdx.x) * 2 * c.N;
    for (int j = threadIdx.y * blockDim.x + threadIdx.x; j < 2 * c.N; j += blockDim.x * blockDim.y) to[j] = joined[j];
}

// Wide rows: dx by itself, reading the row twice.
template <typename T, int V>
__global__ void __launch_bounds__(MOST_THREADS) backward_wide_kernel(const __grid_constant__ Backward c) {
    using R = Row<T, V>;
    using Num = typename R::Num;
    __shared__ __align__(16) float part[2][MOST_WARPS][4];
    const long long r = blockIdx.x;
    tc::grid_trigger();
    tc::grid_wait();
    const T *wp = static_cast<const T *>(c.weight);
    const T *xr = static_cast<const T *>(c.x) + r * c.ldx, *gr = static_cast<const T *>(c.dy) + r * c.lddy;
    const float rstd = c.stats[2 * r + 1];
    const Num minus_mean = all<Num>(-c.stats[2 * r]);
    int turn = 0;
    Num sg = all<Num>(0.0f), sgd = sg, sd = sg;
    // Packs of a thread that are loaded together.  (More in 16 bits cost the SM its blocks:
    // 3000 x 14001 279 us for 180; in FP32 1000 x 16384 91 for 98.)
    constexpr int AT_ONCE = sizeof(T) == 2 ? 2 : 8 / V;
    const auto each = [&](auto &&take) {
        for (int p0 = threadIdx.x; p0 < c.packs; p0 += AT_ONCE * blockDim.x) {
            Pack<T, V> x[AT_ONCE], g[AT_ONCE], w[AT_ONCE];
#pragma unroll
            for (int u = 0; u < AT_ONCE; ++u) {
                const int p = p0 + u * static_cast<int>(blockDim.x);
                const long long at = static_cast<long long>(p) * V;
                const bool in = p < c.packs;
                x[u] = load_if<T, V>(in, xr + at);
                g[u] = load_if<T, V>(in, gr + at);
                w[u] = load_or_ones<T, V>(in && wp != nullptr, wp + at);
            }
#pragma unroll
            for (int u = 0; u < AT_ONCE; ++u)
                if (p0 + u * static_cast<int>(blockDim.x) < c.packs) take(p0 + u * static_cast<int>(blockDim.x), x[u], g[u], w[u]);
        }
    };
    each([&](int, const Pack<T, V> &x, const Pack<T, V> &g, const Pack<T, V> &w) { R::means(x, g, w, minus_mean, sg, sgd, sd); });
    float q[3] = {sum_of(sg), sum_of(sgd), sum_of(sd)};
    row_sum<false>(q, part, turn);
    const RowMeans m = row_means(q, c.inverse, rstd);
    if (c.rest != nullptr && threadIdx.x == 0) c.rest[r] = m.rest;
    if (c.dx == nullptr) return;
    const Num n_rstd = all<Num>(rstd), a = all<Num>(m.a), b = all<Num>(m.b);
    T *dx = static_cast<T *>(c.dx) + r * c.lddx;
    each([&](int p, const Pack<T, V> &x, const Pack<T, V> &g, const Pack<T, V> &w) {
        Num unused_w[R::L::N], unused_b[R::L::N];
#pragma unroll
        for (int k = 0; k < R::L::N; ++k) unused_w[k] = unused_b[k] = all<Num>(0.0f);
        store<T, V>(dx + static_cast<long long>(p) * V,
                    R::gradient(x, g, w, minus_mean, n_rstd, all<Num>(0.0f), a, b, unused_w, unused_b));
    });
}

// Wide rows: the column sums by themselves.  A block takes 32 columns and every
// blocks-th group of 8 rows; its warps' sums are joined in their order.
template <typename T>
__global__ void __launch_bounds__(256) columns_kernel(const __grid_constant__ Backward c) {
    __shared__ float part[2][8][32];
    const int j = blockIdx.x * 32 + threadIdx.x;
    tc::grid_trigger();
    tc::grid_wait();
    float dw = 0.0f, db = 0.0f;
    if (j < c.N)
        for (long long r = static_cast<long long>(blockIdx.y) * 8 + threadIdx.y; r < c.M; r += static_cast<long long>(c.blocks) * 8) {
            const float x = to_f(static_cast<const T *>(c.x)[r * c.ldx + j]), g = to_f(static_cast<const T *>(c.dy)[r * c.lddy + j]);
            dw = fmaf(g, (x - c.stats[2 * r] - c.rest[r]) * c.stats[2 * r + 1], dw);
            db += g;
        }
    part[0][threadIdx.y][threadIdx.x] = dw;
    part[1][threadIdx.y][threadIdx.x] = db;
    __syncthreads();
    if (threadIdx.y < 2 && j < c.N) {
        float t = 0.0f;
#pragma unroll
        for (int y = 0; y < 8; ++y) t += part[threadIdx.y][y][threadIdx.x];
        c.sums[(static_cast<long long>(blockIdx.y) * 2 + threadIdx.y) * c.N + j] = t;
    }
}

// dweight and dbias from the blocks' sums: 32 columns a block, warp y adds
// blocks y, y + 32, ...
template <typename T>
__global__ void __launch_bounds__(1024) join_kernel(const float *__restrict__ sums, int blocks, int N, T *dweight, T *dbias) {
    __shared__ float part[32][33];
    const int j = blockIdx.x * 32 + threadIdx.x, which = blockIdx.y;
    T *to = which == 0 ? dweight : dbias;
    tc::grid_trigger();
    tc::grid_wait();
    if (to == nullptr) return;
    float t = 0.0f;
    if (j < N) {
#pragma unroll 8
        for (int b = threadIdx.y; b < blocks; b += 32) t += sums[(static_cast<long long>(b) * 2 + which) * N + j];
    }
    part[threadIdx.y][threadIdx.x] = t;
    __syncthreads();
    t = part[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) t += __shfl_xor_sync(0xffffffffu, t, k);
    const int col = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && col < N) to[col] = from_f<T>(t);
}

// ---- host ----------------------------------------------------------------------------
constexpr int SMS = 152;
constexpr int WIDE_BLOCKS = 32;            // row groups of columns_kernel
constexpr size_t ROOM = 226 * 1024;        // of shared memory, for rows on their way, weights and joined sums
constexpr size_t SHARED = 171 * 1024;      // of an SM's shared memory, what allow_room's division gives several blocks

int round32(int v) { return (v + 31) / 32 * 32; }

// Rows that a block of MANY_THREADS has threads for (and named barriers, where a row is not a warp's).
int rows_at_once(int packs, int ppt) {
    const int threads = round32((packs + ppt - 1) / ppt), rows = MANY_THREADS / threads;
    return rows > 15 && threads > 32 ? 15 : rows;
}
// Blocks of the gradient, at most: one an SM (the workspace holds the sums of each).
int backward_blocks(int M) { return M < SMS ? M : SMS; }
// The kernel may have `bytes` of shared memory, and (several: more blocks than SMs) an
// SM's is divided so that all the blocks that its registers allow have theirs.
template <typename K>
bool allow_room(K kernel, size_t bytes, bool several) {
    return (bytes <= 40 * 1024 || cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(ROOM)) == cudaSuccess) &&
           (!several || cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 75) == cudaSuccess);
}
size_t up256(size_t b) { return (b + 255) / 256 * 256; }

int check(int type, int M, int N) {
    if (type < LINEAR_F32 || type > LINEAR_F16) return SGEMM_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || M > INT_MAX - 1024 || N > INT_MAX - 65536) return SGEMM_ERR_INVALID_DIM;
    return SGEMM_OK;
}

}  // namespace

extern "C" int layer_norm_forward(int type, int M, int N, const void *x, int64_t ldx, const void *weight, const void *bias,
                                  float eps, float *stats, void *y, int64_t ldy, cudaStream_t stream) {
    const int st = check(type, M, N);
    if (st != SGEMM_OK) return st;
    if (!(eps >= 0.0f) || std::isinf(eps)) return SGEMM_ERR_INVALID_ARG;
    const int least = N > 1 ? N : 1, b = lt::type_bytes(type);
    if (ldx < least || ldy < least) return SGEMM_ERR_INVALID_LD;
    if (M == 0) return SGEMM_OK;
    if (N > 0 && (x == nullptr || y == nullptr)) return SGEMM_ERR_NULL_PTR;
    if (misaligned(x, b) || misaligned(weight, b) || misaligned(bias, b) || misaligned(y, b) || misaligned(stats, 4))
        return SGEMM_ERR_INVALID_ARG;
    const Span out[2] = {span(y, M, N, ldy, b), span(stats, 1, 2LL * M, 2LL * M, 4)};
    const Span in[3] = {span(x, M, N, ldx, b), span(weight, 1, N, N, b), span(bias, 1, N, N, b)};
    for (const Span &o : out)
        for (const Span &i : in)
            if (overlap(o, i)) return SGEMM_ERR_ALIAS;
    if (overlap(out[0], out[1])) return SGEMM_ERR_ALIAS;
    if (N == 0) return stats == nullptr ? SGEMM_OK : launched(cudaMemsetAsync(stats, 0, sizeof(float) * 2 * static_cast<size_t>(M), stream));
    Forward c{};
    c.x = x, c.weight = weight, c.bias = bias, c.y = y, c.stats = stats, c.ldx = ldx, c.ldy = ldy, c.M = M, c.N = N, c.eps = eps;
    c.inverse = 1.0f / static_cast<float>(N);
    const int width = narrower(narrower(width_of(x, ldx, type), width_of(y, ldy, type)),
                               narrower(narrower(width_of(weight, 0, type), width_of(bias, 0, type)), width_of(x, N, type)));
    c.packs = N / (width / b);
    sg_nvtx::Range r("layer norm");
    return with_rows(type, width, [&](auto el, auto v) {
        using El = decltype(el);
        constexpr int V = decltype(v)::value;
        constexpr int BYTES = V * static_cast<int>(sizeof(El));
        auto run = [&](auto kernel, int ppt, int block) {
            const int threads = round32((c.packs + ppt - 1) / ppt), rows = threads == 32 ? 4 : 1;
            const long long groups = (static_cast<long long>(M) + rows - 1) / rows;
            const size_t room = BYTES >= 4 ? static_cast<size_t>(2) * ppt * block * BYTES : 0;
            // all blocks at once: each has its rows from the start
            long long most = threads * rows <= 1024 ? 1024 / (threads * rows) : 1;
            const long long rooms = static_cast<long long>(SHARED / (room + 2048));
            if (most > rooms) most = rooms;
            most *= SMS;
            if (!allow_room(kernel, room, groups > SMS)) return static_cast<int>(SGEMM_ERR_DEVICE);
            return launched(tc::launch(kernel, static_cast<unsigned>(groups < most ? groups : most), dim3(threads, rows), room, stream, c));
        };
        // Of rows longer than a warp's, 16 values (one by one: 8) or 32 (16) a thread, what has
        // more rows at once.  Two blocks an SM where that is one and the packs are 16 bytes
        // (3000 x 14336 bf16 39 us for 46), or where weight and bias have no room (FP32).  FP32
        // by 8 bytes: 16 values (8188 x 4098 57 us, 32 values 70).
        constexpr int LARGE = V > 1 ? 32 / V : 16, SMALL = LARGE / 4;
        if (c.packs <= SMALL * 32) return run(forward_kernel<El, V, SMALL, 128, false>, SMALL, 128);
        const int few = rows_at_once(c.packs, LARGE / 2), many = rows_at_once(c.packs, LARGE);
        const size_t slots = BYTES >= 4 ? static_cast<size_t>(2) * MANY_THREADS * BYTES : 0, weights = static_cast<size_t>(2) * c.packs * BYTES;
        constexpr bool MANY = sizeof(El) == 2 || V != 2;
        const bool many_fit = MANY && weights + LARGE * slots <= ROOM, few_fit = weights + LARGE / 2 * slots <= ROOM;
        if constexpr (BYTES == 16 || (sizeof(El) == 4 && V > 1))
            if (c.packs <= LARGE * MOST_THREADS && (BYTES == 16 ? many <= 1 : !many_fit && (few == 0 || !few_fit)))
                return run(forward_kernel<El, V, LARGE, MOST_THREADS, false>, LARGE, MOST_THREADS);
        auto several = [&](auto kernel, int ppt, int rows) {
            if (rows > (M + SMS - 1) / SMS) rows = (M + SMS - 1) / SMS;
            const long long groups = (static_cast<long long>(M) + rows - 1) / rows;
            const size_t room = weights + ppt * slots;
            if (!allow_room(kernel, room, false)) return static_cast<int>(SGEMM_ERR_DEVICE);
            return launched(tc::launch(kernel, static_cast<unsigned>(groups < SMS ? groups : SMS),
                                       dim3(round32((c.packs + ppt - 1) / ppt), rows), room, stream, c));
        };
        if constexpr (MANY)
            if (many > few && many_fit) return several(forward_kernel<El, V, LARGE, MANY_THREADS, true>, LARGE, many);
        if (few > 0 && few_fit) return several(forward_kernel<El, V, LARGE / 2, MANY_THREADS, true>, LARGE / 2, few);
        return launched(tc::launch(forward_wide_kernel<El, V>, static_cast<unsigned>(M), dim3(MOST_THREADS), 0, stream, c));
    });
}

extern "C" size_t layer_norm_backward_workspace_size(int M, int N, int want_dweight, int want_dbias) {
    if (M <= 0 || N <= 0 || !(want_dweight || want_dbias)) return 0;
    const int blocks = backward_blocks(M);
    return up256(sizeof(float) * 2 * static_cast<size_t>(blocks) * N) + up256(sizeof(float) * static_cast<size_t>(M));
}

extern "C" int layer_norm_backward(int type, int M, int N, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                   const void *weight, const float *stats, void *dx, int64_t lddx, void *dweight, void *dbias,
                                   void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    const int st = check(type, M, N);
    if (st != SGEMM_OK) return st;
    const int least = N > 1 ? N : 1, b = lt::type_bytes(type);
    if (lddy < least || ldx < least || (dx != nullptr && lddx < least)) return SGEMM_ERR_INVALID_LD;
    if (N == 0 || (dx == nullptr && dweight == nullptr && dbias == nullptr)) return SGEMM_OK;
    if (M > 0 && (dy == nullptr || x == nullptr || stats == nullptr)) return SGEMM_ERR_NULL_PTR;
    const size_t need = layer_norm_backward_workspace_size(M, N, dweight != nullptr, dbias != nullptr);
    if (need > 0 && workspace == nullptr) return SGEMM_ERR_NULL_PTR;
    if (misaligned(dy, b) || misaligned(x, b) || misaligned(weight, b) || misaligned(stats, 4) || misaligned(dx, b) ||
        misaligned(dweight, b) || misaligned(dbias, b) || misaligned(workspace, 256) || workspace_bytes < need)
        return SGEMM_ERR_INVALID_ARG;
    const Span out[4] = {span(dx, M, N, lddx, b), span(dweight, 1, N, N, b), span(dbias, 1, N, N, b),
                         span(workspace, 1, static_cast<long long>(need), 1, 1)};
    const Span in[4] = {span(dy, M, N, lddy, b), span(x, M, N, ldx, b), span(weight, 1, N, N, b),
                        span(stats, 1, 2LL * M, 2LL * M, 4)};
    for (int i = 0; i < 4; ++i) {
        for (const Span &s : in)
            if (overlap(out[i], s)) return SGEMM_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return SGEMM_ERR_ALIAS;
    }
    const size_t column = static_cast<size_t>(N) * b;
    if (M == 0) {
        cudaError_t err = dweight != nullptr ? cudaMemsetAsync(dweight, 0, column, stream) : cudaSuccess;
        if (err == cudaSuccess && dbias != nullptr) err = cudaMemsetAsync(dbias, 0, column, stream);
        return launched(err);
    }
    const bool columns = dweight != nullptr || dbias != nullptr;
    Backward c{};
    c.dy = dy, c.x = x, c.weight = weight, c.stats = stats, c.dx = dx, c.dweight = dweight, c.dbias = dbias;
    c.lddy = lddy, c.ldx = ldx, c.lddx = lddx, c.M = M, c.N = N;
    c.inverse = 1.0f / static_cast<float>(N);
    c.blocks = backward_blocks(M);
    if (columns) {
        c.sums = static_cast<float *>(workspace);
        c.rest = reinterpret_cast<float *>(static_cast<char *>(workspace) + up256(sizeof(float) * 2 * static_cast<size_t>(c.blocks) * N));
    }
    const int width = narrower(narrower(width_of(dy, lddy, type), width_of(x, ldx, type)),
                               narrower(narrower(width_of(dx, lddx, type), width_of(weight, 0, type)), width_of(x, N, type)));
    c.packs = N / (width / b);
    sg_nvtx::Range r("layer norm: backward");
    const int done = with_rows(type, width, [&](auto el, auto v) {
        using El = decltype(el);
        constexpr int V = decltype(v)::value;
        constexpr int BYTES = V * static_cast<int>(sizeof(El));
        auto run = [&](auto kernel, int ppt, int block, size_t room) {
            const int threads = round32((c.packs + ppt - 1) / ppt);
            int rows = block / threads;
            if (rows > 15 && threads > 32) rows = 15;  // named barriers
            const int groups = static_cast<int>((static_cast<long long>(M) + rows - 1) / rows);
            if (groups < c.blocks) c.blocks = groups;
            if (!allow_room(kernel, room, false)) return static_cast<int>(SGEMM_ERR_DEVICE);
            return launched(tc::launch(kernel, static_cast<unsigned>(c.blocks), dim3(threads, rows), room, stream, c));
        };
        // 16 values of a row a thread (one by one: 8), or twice as many of a wide one where registers and room allow
        constexpr int SMALL = V > 1 ? 16 / V : 8, LARGE = 2 * SMALL;
        auto room_of = [&](int ppt, int block, bool weight) {
            const size_t slots = BYTES >= 4 ? static_cast<size_t>(4) * ppt * block * BYTES : 0, sums = sizeof(float) * 2 * static_cast<size_t>(N);
            const size_t rows = slots + (weight ? static_cast<size_t>(c.packs) * BYTES : 0);
            return rows > sums ? rows : sums;
        };
        constexpr bool SHARED_WEIGHT = BYTES != 4 || sizeof(El) == 2;
        if (c.packs <= SMALL * MANY_THREADS) {
            const size_t room = room_of(SMALL, MANY_THREADS, SHARED_WEIGHT);
            // (a lane's one pack of weights comes sooner from L1: 400000 x 128 bf16 122 us for 150, 60000 x 256 29.6
            // for 33.5; not so where it has more, or in FP32: 60000 x 512 bf16 48.7 for 45.4, 60000 x 128 f32 24.8 for 22.8)
            if constexpr (SHARED_WEIGHT && (sizeof(El) == 4 || BYTES == 16))
                if (room > ROOM || (sizeof(El) == 2 && c.packs <= 32))
                    return run(backward_kernel<El, V, SMALL, MANY_THREADS, false>, SMALL, MANY_THREADS, room_of(SMALL, MANY_THREADS, false));
            return run(backward_kernel<El, V, SMALL, MANY_THREADS, SHARED_WEIGHT>, SMALL, MANY_THREADS, room);
        }
        if constexpr (sizeof(El) == 2 || V == 1) {
            constexpr int BLOCK = sizeof(El) == 4 ? MANY_THREADS : MOST_THREADS;
            if (c.packs <= LARGE * BLOCK)
                return run(backward_kernel<El, V, LARGE, BLOCK, SHARED_WEIGHT>, LARGE, BLOCK, room_of(LARGE, BLOCK, SHARED_WEIGHT));
        }
        int s = launched(tc::launch(backward_wide_kernel<El, V>, static_cast<unsigned>(M), dim3(MOST_THREADS), 0, stream, c));
        if (s == SGEMM_OK && columns) {
            c.blocks = c.blocks < WIDE_BLOCKS ? c.blocks : WIDE_BLOCKS;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>((N + 31) / 32), static_cast<unsigned>(c.blocks));
            cfg.blockDim = dim3(32, 8);
            cfg.stream = stream;
            s = launched(cudaLaunchKernelEx(&cfg, columns_kernel<El>, c));
        }
        return s;
    });
    if (done != SGEMM_OK || !columns) return done;
    auto join = [&](auto el) {
        using El = decltype(el);
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3(static_cast<unsigned>((N + 31) / 32), 2);
        cfg.blockDim = dim3(32, 32);
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return launched(cudaLaunchKernelEx(&cfg, join_kernel<El>, static_cast<const float *>(c.sums), c.blocks, N, static_cast<El *>(dweight),
                                           static_cast<El *>(dbias)));
    };
    return type == LINEAR_F32 ? join(float()) : type == LINEAR_BF16 ? join(__nv_bfloat16()) : join(__half());
}
