// norm.cu -- layer norm and its gradient (C ABI: include/norm.h).  Bound by
// HBM: the forward pass reads and writes each value once, the gradient reads
// two and writes one.
//
// A row is held in the registers of `threads` threads (a warp, or a block) while
// its sums go round: thread k has packs k, k + threads, ... of V values.  The
// mean is rounded; the differences to it are summed again, which gives what the
// rounding left, and squared for the variance, which so has no cancellation.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "linear_types.cuh"
#include "norm.h"
#include "nvtx_range.cuh"
#include "rows.cuh"
#include "tensor_core.cuh"

namespace {

using namespace rows;

constexpr int WARP_ROWS = 4;       // rows of a block, if a warp holds one
constexpr int MOST_THREADS = 1024;

// The sums of N values over the threads of a row (blockDim.x of them), the same
// in each: across the warp, then over the warps in their order.  `part` has two
// sets, used in turn (`turn`), so that one barrier a sum is enough.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*part)[32][4], int &turn) {
#pragma unroll
    for (int k = 16; k > 0; k >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], k);
    if (blockDim.x == 32) return;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) part[turn][threadIdx.x >> 5][i] = v[i];
    __syncthreads();
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane < warps ? part[turn][lane][i] : 0.0f;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], k);
    turn ^= 1;
}

struct Forward {
    const void *x, *weight, *bias;
    void *y;
    float *stats;
    long long ldx, ldy;
    int M, N, packs;
    float eps;
};

template <typename T, int V>
__device__ __forceinline__ void finish(const Pack<T, V> &x, const Pack<T, V> &w, const Pack<T, V> &b, bool has_w, float mean,
                                       float rest, float rstd, T *y) {
    float f[V], fw[V], fb[V];
    x.get(f);
    w.get(fw);
    b.get(fb);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const float h = (f[k] - mean - rest) * rstd;
        f[k] = fmaf(h, has_w ? fw[k] : 1.0f, fb[k]);
    }
    Pack<T, V> o;
    o.set(f);
    store<T, V>(y, o);
}

// PPT packs a thread.
template <typename T, int V, int PPT>
__global__ void __launch_bounds__(MOST_THREADS) forward_kernel(const __grid_constant__ Forward c) {
    __shared__ float part[2][32][4];
    const long long r = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    tc::grid_trigger();
    tc::grid_wait();
    if (r >= c.M) return;
    const T *row = static_cast<const T *>(c.x) + r * c.ldx;
    const T *wp = static_cast<const T *>(c.weight), *bp = static_cast<const T *>(c.bias);
    Pack<T, V> x[PPT], w[PPT], b[PPT];
    int turn = 0;
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
        const int p = threadIdx.x + i * blockDim.x;
        x[i] = load_if<T, V>(p < c.packs, row + static_cast<long long>(p) * V);
        w[i] = load_if<T, V>(p < c.packs && wp != nullptr, wp + static_cast<long long>(p) * V);
        b[i] = load_if<T, V>(p < c.packs && bp != nullptr, bp + static_cast<long long>(p) * V);
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
        float f[V];
        x[i].get(f);
#pragma unroll
        for (int k = 0; k < V; ++k) s[0] += f[k];
    }
    row_sum(s, part, turn);
    const float mean = s[0] / static_cast<float>(c.N);
    float q[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
        float f[V];
        x[i].get(f);
        if (threadIdx.x + i * blockDim.x < c.packs)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float d = f[k] - mean;
                q[0] += d;
                q[1] = fmaf(d, d, q[1]);
            }
    }
    row_sum(q, part, turn);
    const float rest = q[0] / static_cast<float>(c.N);
    const float var = fmaf(-rest, rest, q[1] / static_cast<float>(c.N));
    const float rstd = 1.0f / sqrtf(fmaxf(var, 0.0f) + c.eps);
    if (c.stats != nullptr && threadIdx.x == 0) {
        c.stats[2 * r] = mean + rest;
        c.stats[2 * r + 1] = rstd;
    }
    T *y = static_cast<T *>(c.y) + r * c.ldy;
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
        const int p = threadIdx.x + i * blockDim.x;
        if (p < c.packs) finish<T, V>(x[i], w[i], b[i], wp != nullptr, mean, rest, rstd, y + static_cast<long long>(p) * V);
    }
}

// Rows that no block's registers hold: read three times, the later ones from L2.
template <typename T, int V>
__global__ void __launch_bounds__(MOST_THREADS) forward_wide_kernel(const __grid_constant__ Forward c) {
    __shared__ float part[2][32][4];
    const long long r = blockIdx.x;
    tc::grid_trigger();
    tc::grid_wait();
    const T *row = static_cast<const T *>(c.x) + r * c.ldx;
    const T *wp = static_cast<const T *>(c.weight), *bp = static_cast<const T *>(c.bias);
    int turn = 0;
    float s[1] = {0.0f};
#pragma unroll 4
    for (int p = threadIdx.x; p < c.packs; p += blockDim.x) {
        float f[V];
        load<T, V>(row + static_cast<long long>(p) * V).get(f);
#pragma unroll
        for (int k = 0; k < V; ++k) s[0] += f[k];
    }
    row_sum(s, part, turn);
    const float mean = s[0] / static_cast<float>(c.N);
    float q[2] = {0.0f, 0.0f};
#pragma unroll 4
    for (int p = threadIdx.x; p < c.packs; p += blockDim.x) {
        float f[V];
        load<T, V>(row + static_cast<long long>(p) * V).get(f);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float d = f[k] - mean;
            q[0] += d;
            q[1] = fmaf(d, d, q[1]);
        }
    }
    row_sum(q, part, turn);
    const float rest = q[0] / static_cast<float>(c.N);
    const float var = fmaf(-rest, rest, q[1] / static_cast<float>(c.N));
    const float rstd = 1.0f / sqrtf(fmaxf(var, 0.0f) + c.eps);
    if (c.stats != nullptr && threadIdx.x == 0) {
        c.stats[2 * r] = mean + rest;
        c.stats[2 * r + 1] = rstd;
    }
    T *y = static_cast<T *>(c.y) + r * c.ldy;
#pragma unroll 4
    for (int p = threadIdx.x; p < c.packs; p += blockDim.x) {
        const long long at = static_cast<long long>(p) * V;
        finish<T, V>(load<T, V>(row + at), load_if<T, V>(wp != nullptr, wp + at), load_if<T, V>(bp != nullptr, bp + at),
                     wp != nullptr, mean, rest, rstd, y + at);
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
};

// Of a row: the sums of g, of g d and of d (d = x - mean) give, with rest = mean of d,
// the two means that dx needs.
struct RowMeans {
    float rest, g, gh;
};
__device__ __forceinline__ RowMeans row_means(const float (&q)[3], float n, float rstd) {
    RowMeans m;
    m.rest = q[2] / n;
    m.g = q[0] / n;
    m.gh = (q[1] / n - m.rest * m.g) * rstd;
    return m;
}

// A grid of `blocks` blocks takes the rows in turn; a thread keeps the sums of
// its columns in registers and writes them at the end.
template <typename T, int V, int PPT, int THREADS>
__global__ void __launch_bounds__(THREADS) backward_kernel(const __grid_constant__ Backward c) {
    __shared__ float part[2][32][4];
    extern __shared__ float joined[];  // WARP_ROWS warps' sums
    float dw[PPT][V], db[PPT][V];
#pragma unroll
    for (int i = 0; i < PPT; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) dw[i][k] = db[i][k] = 0.0f;
    tc::grid_trigger();
    tc::grid_wait();
    const T *wp = static_cast<const T *>(c.weight);
    const float n = static_cast<float>(c.N);
    int turn = 0;
    for (long long r = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y; r < c.M;
         r += static_cast<long long>(c.blocks) * blockDim.y) {
        const T *xr = static_cast<const T *>(c.x) + r * c.ldx, *gr = static_cast<const T *>(c.dy) + r * c.lddy;
        Pack<T, V> x[PPT], g[PPT];
#pragma unroll
        for (int i = 0; i < PPT; ++i) {
            const int p = threadIdx.x + i * blockDim.x;
            x[i] = load_if<T, V>(p < c.packs, xr + static_cast<long long>(p) * V);
            g[i] = load_if<T, V>(p < c.packs, gr + static_cast<long long>(p) * V);
        }
        const float mean = c.stats[2 * r], rstd = c.stats[2 * r + 1];
        float q[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < PPT; ++i) {
            const int p = threadIdx.x + i * blockDim.x;
            if (p < c.packs) {
                float fx[V], fg[V], fw[V];
                x[i].get(fx);
                g[i].get(fg);
                load_if<T, V>(wp != nullptr, wp + static_cast<long long>(p) * V).get(fw);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float d = fx[k] - mean, gw = wp != nullptr ? fg[k] * fw[k] : fg[k];
                    q[0] += gw;
                    q[1] = fmaf(gw, d, q[1]);
                    q[2] += d;
                }
            }
        }
        row_sum(q, part, turn);
        const RowMeans m = row_means(q, n, rstd);
        T *dx = static_cast<T *>(c.dx) + r * c.lddx;
#pragma unroll
        for (int i = 0; i < PPT; ++i) {
            const int p = threadIdx.x + i * blockDim.x;
            if (p < c.packs) {
                float fx[V], fg[V], fw[V];
                x[i].get(fx);
                g[i].get(fg);
                load_if<T, V>(wp != nullptr, wp + static_cast<long long>(p) * V).get(fw);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float h = (fx[k] - mean - m.rest) * rstd;
                    dw[i][k] = fmaf(fg[k], h, dw[i][k]);
                    db[i][k] += fg[k];
                    const float gw = wp != nullptr ? fg[k] * fw[k] : fg[k];
                    fx[k] = rstd * (gw - m.g - h * m.gh);
                }
                if (c.dx != nullptr) {
                    Pack<T, V> o;
                    o.set(fx);
                    store<T, V>(dx + static_cast<long long>(p) * V, o);
                }
            }
        }
    }
    if (c.sums == nullptr) return;
    float *to = c.sums + static_cast<long long>(blockIdx.x) * 2 * c.N;
    if (blockDim.y > 1) {  // the warps' sums, in their order
        for (int s = 0; s < 2; ++s) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < PPT; ++i) {
                const int p = threadIdx.x + i * 32;
                if (p < c.packs)
#pragma unroll
                    for (int k = 0; k < V; ++k) joined[threadIdx.y * c.N + p * V + k] = s == 0 ? dw[i][k] : db[i][k];
            }
            __syncthreads();
            for (int j = threadIdx.y * 32 + threadIdx.x; j < c.N; j += blockDim.y * 32) {
                float t = 0.0f;
                for (int y = 0; y < static_cast<int>(blockDim.y); ++y) t += joined[y * c.N + j];
                to[s * static_cast<long long>(c.N) + j] = t;
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < PPT; ++i) {
        const int p = threadIdx.x + i * blockDim.x;
        if (p < c.packs)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                to[static_cast<long long>(p) * V + k] = dw[i][k];
                to[c.N + static_cast<long long>(p) * V + k] = db[i][k];
            }
    }
}

// Wide rows: dx by itself, reading the row twice.
template <typename T, int V>
__global__ void __launch_bounds__(MOST_THREADS) backward_wide_kernel(const __grid_constant__ Backward c) {
    __shared__ float part[2][32][4];
    const long long r = blockIdx.x;
    tc::grid_trigger();
    tc::grid_wait();
    const T *wp = static_cast<const T *>(c.weight);
    const T *xr = static_cast<const T *>(c.x) + r * c.ldx, *gr = static_cast<const T *>(c.dy) + r * c.lddy;
    const float mean = c.stats[2 * r], rstd = c.stats[2 * r + 1];
    int turn = 0;
    float q[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll 2
    for (int p = threadIdx.x; p < c.packs; p += blockDim.x) {
        const long long at = static_cast<long long>(p) * V;
        float fx[V], fg[V], fw[V];
        load<T, V>(xr + at).get(fx);
        load<T, V>(gr + at).get(fg);
        load_if<T, V>(wp != nullptr, wp + at).get(fw);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float d = fx[k] - mean, gw = wp != nullptr ? fg[k] * fw[k] : fg[k];
            q[0] += gw;
            q[1] = fmaf(gw, d, q[1]);
            q[2] += d;
        }
    }
    row_sum(q, part, turn);
    const RowMeans m = row_means(q, static_cast<float>(c.N), rstd);
    if (c.rest != nullptr && threadIdx.x == 0) c.rest[r] = m.rest;
    if (c.dx == nullptr) return;
    T *dx = static_cast<T *>(c.dx) + r * c.lddx;
#pragma unroll 2
    for (int p = threadIdx.x; p < c.packs; p += blockDim.x) {
        const long long at = static_cast<long long>(p) * V;
        float fx[V], fg[V], fw[V];
        load<T, V>(xr + at).get(fx);
        load<T, V>(gr + at).get(fg);
        load_if<T, V>(wp != nullptr, wp + at).get(fw);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float h = (fx[k] - mean - m.rest) * rstd, gw = wp != nullptr ? fg[k] * fw[k] : fg[k];
            fx[k] = rstd * (gw - m.g - h * m.gh);
        }
        Pack<T, V> o;
        o.set(fx);
        store<T, V>(dx + at, o);
    }
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
#pragma unroll 4
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
constexpr int MOST_BLOCKS = 2 * SMS;  // of the gradient: their sums are written and read once more
constexpr int WIDE_BLOCKS = 32;       // row groups of columns_kernel
constexpr int BACKWARD_THREADS = 512;

int round32(int v) { return (v + 31) / 32 * 32; }

// How the gradient's grid shares the rows out, from sizes alone (the workspace depends on it).
int backward_blocks(int M, int N) {
    const int rows = N <= 1024 ? WARP_ROWS : 1;
    const long long groups = (static_cast<long long>(M) + rows - 1) / rows;
    return static_cast<int>(groups < MOST_BLOCKS ? groups : MOST_BLOCKS);
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
    const int width = narrower(narrower(width_of(x, ldx, type), width_of(y, ldy, type)),
                               narrower(narrower(width_of(weight, 0, type), width_of(bias, 0, type)), width_of(x, N, type)));
    c.packs = N / (width / b);
    sg_nvtx::Range r("layer norm");
    return with_rows(type, width, [&](auto el, auto v) {
        using El = decltype(el);
        constexpr int V = decltype(v)::value;
        auto run = [&](auto kernel, int ppt) {
            const int threads = round32((c.packs + ppt - 1) / ppt), rows = threads == 32 ? WARP_ROWS : 1;
            return launched(tc::launch(kernel, static_cast<unsigned>((M + rows - 1) / rows), dim3(threads, rows), 0, stream, c));
        };
        constexpr int SMALL = V >= 8 ? 2 : 4, LARGE = V >= 8 ? 4 : V == 1 ? 16 : 32 / V;
        if (c.packs <= SMALL * 128) return run(forward_kernel<El, V, SMALL>, SMALL);
        if (c.packs <= LARGE * MOST_THREADS) return run(forward_kernel<El, V, LARGE>, LARGE);
        return launched(tc::launch(forward_wide_kernel<El, V>, static_cast<unsigned>(M), dim3(MOST_THREADS), 0, stream, c));
    });
}

extern "C" size_t layer_norm_backward_workspace_size(int M, int N, int want_dweight, int want_dbias) {
    if (M <= 0 || N <= 0 || !(want_dweight || want_dbias)) return 0;
    const int blocks = backward_blocks(M, N);
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
    c.blocks = backward_blocks(M, N);
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
        auto run = [&](auto kernel, int ppt) {
            const int threads = round32((c.packs + ppt - 1) / ppt);
            const int rows = threads == 32 && N <= 1024 ? WARP_ROWS : 1;
            const size_t smem = rows > 1 && columns ? sizeof(float) * WARP_ROWS * static_cast<size_t>(N) : 0;
            return launched(tc::launch(kernel, static_cast<unsigned>(c.blocks), dim3(threads, rows), smem, stream, c));
        };
        constexpr int SMALL = V >= 8 ? 2 : 4, LARGE = V >= 8 ? 4 : V >= 4 ? 4 : 16;
        if (c.packs <= SMALL * 256) return run(backward_kernel<El, V, SMALL, 256>, SMALL);
        if (c.packs <= LARGE * BACKWARD_THREADS) return run(backward_kernel<El, V, LARGE, BACKWARD_THREADS>, LARGE);
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
