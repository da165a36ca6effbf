// experts.cu -- the tokens' way to their experts and back (C ABI:
// include/experts.h).  Everything here moves bytes: a stable counting sort of
// the choices, and copies and sums of whole rows in 16-byte accesses where
// the rows allow it, one 16-byte column per thread so that each row of x, y
// and dy is read or written once.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <type_traits>

#include "experts.h"
#include "linear_types.cuh"
#include "nvtx_range.cuh"
#include "tensor_core.cuh"

namespace {

using lt::from_f;
using lt::to_f;

// ---- sort ------------------------------------------------------------------------
// Choices are cut into `blocks` equal ranges.  With more than one, a first
// kernel counts each range's choices by expert; the second adds up what lies
// before its range, counts its own range warp by warp and gives each choice
// its place: places before the expert + before the range + before the warp +
// in the warp.  Nothing there depends on which thread runs first, so the order is
// that of the choices; only the ranges' counts are added up by atomics, and sums
// of whole numbers are the same in any order.
constexpr int SORT_THREADS = 1024;
constexpr int SORT_ALONE = 4096;   // choices that one block sorts in one launch
constexpr int SORT_RANGE = 1024;   // choices of a block, with more: one step of its 32 warps
constexpr int SORT_BLOCKS = 256;   // ranges, at most: each block reads all their counts
constexpr int SORT_SMEM = 200 * 1024;

struct SortPlan {
    int blocks, range, warps;
    size_t smem;
};
SortPlan sort_plan(long long R, int E) {
    SortPlan s;
    long long blocks = R <= SORT_ALONE ? 1 : (R + SORT_RANGE - 1) / SORT_RANGE;
    if (blocks > SORT_BLOCKS) blocks = SORT_BLOCKS;
    s.range = static_cast<int>(((R + blocks - 1) / blocks + 31) / 32 * 32);
    if (s.range < 32) s.range = 32;
    s.blocks = static_cast<int>((R + s.range - 1) / s.range);
    if (s.blocks < 1) s.blocks = 1;
    const int most = SORT_SMEM / 4 / E - 3;  // tables of E counts that fit, beside three for all warps
    s.warps = most < SORT_THREADS / 32 ? most : SORT_THREADS / 32;
    s.smem = static_cast<size_t>(s.warps + 3) * E * 4;
    return s;
}

template <typename I>
__device__ __forceinline__ int choice_at(const I *choices, long long i, long long end, int E) {
    if (i >= end) return -1;
    const I c = choices[i];
    return c >= 0 && c < E ? static_cast<int>(c) : -1;
}
// Adds 32 choices (one per lane, -1: none) to a warp's counts; returns each
// one's place among its expert's (before: what the counts held).
__device__ __forceinline__ int count32(int key, int *counts, int lane) {
    const unsigned same = __match_any_sync(0xffffffffu, key);
    int before = 0;
    if (key >= 0) before = counts[key];
    __syncwarp();
    if (key >= 0 && lane == __ffs(same) - 1) counts[key] = before + __popc(same);
    __syncwarp();
    return before + __popc(same & ((1u << lane) - 1u));
}

template <typename I>
__global__ void __launch_bounds__(SORT_THREADS) sort_count_kernel(const I *__restrict__ choices, long long R, int E,
                                                                  int range, int warps, int *__restrict__ counts) {
    extern __shared__ int shared[];
    tc::grid_wait();
    tc::grid_trigger();  // the second kernel counts its ranges meanwhile (the choices are there now)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < warps * E; i += SORT_THREADS) shared[i] = 0;
    __syncthreads();
    const long long begin = static_cast<long long>(blockIdx.x) * range;
    const long long end = begin + range < R ? begin + range : R;
    const int per = ((range + warps - 1) / warps + 31) / 32 * 32;
    if (warp < warps) {
        const long long b = begin + static_cast<long long>(warp) * per, e = b + per < end ? b + per : end;
        for (long long i = b; i < e; i += 32) count32(choice_at(choices, i + lane, e, E), shared + warp * E, lane);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += SORT_THREADS) {
        int n = 0;
        for (int w = 0; w < warps; ++w) n += shared[w * E + e];
        counts[static_cast<long long>(blockIdx.x) * E + e] = n;
    }
}

template <typename I>
__global__ void __launch_bounds__(SORT_THREADS)
sort_place_kernel(const I *__restrict__ choices, long long R, int E, int range, int warps, int blocks,
                  const int *__restrict__ counts, int *__restrict__ rows, int *__restrict__ offsets) {
    extern __shared__ int shared[];
    __shared__ int sums[32];
    int *base = shared;                  // E: the expert's first place in this range
    int *totals = shared + E;            // E: all its choices
    int *earlier = totals + E;           // E: those in the ranges before this one
    int *mine = earlier + E;             // warps x E
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < (warps + 2) * E; i += SORT_THREADS) totals[i] = 0;
    if (blocks == 1) tc::grid_wait();  // else the first kernel has waited for the choices
    __syncthreads();
    const long long begin = static_cast<long long>(blockIdx.x) * range;
    const long long end = begin + range < R ? begin + range : R;
    const int per = ((range + warps - 1) / warps + 31) / 32 * 32;
    const long long b = begin + static_cast<long long>(warp) * per, e1 = b + per < end ? b + per : end;
    if (warp < warps)
        for (long long i = b; i < e1; i += 32) count32(choice_at(choices, i + lane, e1, E), mine + warp * E, lane);
    __syncthreads();
    tc::grid_wait();  // the counts are there, and rows and offsets no longer in use
    if (blocks > 1) {
        for (int i = threadIdx.x; i < blocks * E; i += SORT_THREADS) {
            const int k = i / E, e = i - k * E, n = counts[i];
            if (n != 0) {  // whole numbers: any order gives the same sums
                atomicAdd(totals + e, n);
                if (k < static_cast<int>(blockIdx.x)) atomicAdd(earlier + e, n);
            }
        }
        __syncthreads();
    }
    // per expert: all its choices, those before this range, and the warps' first places;
    // the running sum over the experts carries from one group of 1024 to the next
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += SORT_THREADS) {
        const int e = e0 + threadIdx.x;
        int total = 0, before = 0;
        if (e < E) {
            int own = 0;
            for (int w = 0; w < warps; ++w) {
                const int n = mine[w * E + e];
                mine[w * E + e] = own;
                own += n;
            }
            total = blocks == 1 ? own : totals[e];
            before = earlier[e];
        }
        int scan = total;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, scan, d);
            if (lane >= d) scan += o;
        }
        if (lane == 31) sums[warp] = scan;
        __syncthreads();
        int ahead = 0, all = 0;
        for (int w = 0; w < SORT_THREADS / 32; ++w) {
            if (w < warp) ahead += sums[w];
            all += sums[w];
        }
        const int first = carry + ahead + scan - total;
        if (e < E) {
            base[e] = first + before;
            if (blockIdx.x == 0) {
                offsets[e] = first;
                if (e == E - 1) offsets[E] = first + total;
            }
        }
        carry += all;
        __syncthreads();
    }
    if (warp < warps)
        for (long long i = b; i < e1; i += 32) {
            const int key = choice_at(choices, i + lane, e1, E);
            const int at = count32(key, mine + warp * E, lane);
            if (i + lane < e1) rows[i + lane] = key >= 0 ? base[key] + at : -1;
        }
}

// ---- rows --------------------------------------------------------------------------
// V values (16, 8, 4 or 2 bytes) of a row, as the word they travel in: a load
// that may not happen is then one predicated instruction, and the next ones
// follow it at once.
template <int BYTES>
struct Word;
template <>
struct Word<16> {
    using type = uint4;
};
template <>
struct Word<8> {
    using type = uint2;
};
template <>
struct Word<4> {
    using type = uint32_t;
};
template <>
struct Word<2> {
    using type = uint16_t;
};
template <typename T, int V>
struct Pack {
    static constexpr int BYTES = V * static_cast<int>(sizeof(T));
    using Raw = typename Word<BYTES>::type;
    Raw raw;
    __device__ __forceinline__ void clear() { raw = Raw{}; }
    __device__ __forceinline__ uint32_t word(int i) const {
        if constexpr (BYTES == 16) return i == 0 ? raw.x : i == 1 ? raw.y : i == 2 ? raw.z : raw.w;
        if constexpr (BYTES == 8) return i == 0 ? raw.x : raw.y;
        if constexpr (BYTES <= 4) return raw;
    }
    __device__ __forceinline__ void get(float (&f)[V]) const {
        if constexpr (BYTES == 2) {
            f[0] = to_f(*reinterpret_cast<const T *>(&raw));
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = __uint_as_float(word(i));
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 v = lt::unpack2<T>(word(i));
                f[2 * i] = v.x;
                f[2 * i + 1] = v.y;
            }
        }
    }
    __device__ __forceinline__ void set(const float (&f)[V]) {
        if constexpr (BYTES == 2) {
            const T v = from_f<T>(f[0]);
            raw = *reinterpret_cast<const Raw *>(&v);
        } else {
            uint32_t w[BYTES / 4];
#pragma unroll
            for (int i = 0; i < BYTES / 4; ++i) {
                if constexpr (sizeof(T) == 4)
                    w[i] = __float_as_uint(f[i]);
                else
                    w[i] = lt::pack2<T>(f[2 * i], f[2 * i + 1]);
            }
            if constexpr (BYTES == 16) raw = make_uint4(w[0], w[1], w[2], w[3]);
            if constexpr (BYTES == 8) raw = make_uint2(w[0], w[1]);
            if constexpr (BYTES == 4) raw = w[0];
        }
    }
};
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load(const T *p) {
    Pack<T, V> v;
    v.raw = *reinterpret_cast<const typename Pack<T, V>::Raw *>(p);
    return v;
}
// The values at p, or zeros.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_if(bool in, const T *p) {
    Pack<T, V> v;
    v.clear();
    if (in) v.raw = *reinterpret_cast<const typename Pack<T, V>::Raw *>(p);
    return v;
}
template <typename T, int V>
__device__ __forceinline__ void store(T *p, const Pack<T, V> &v) {
    *reinterpret_cast<typename Pack<T, V>::Raw *>(p) = v.raw;
}

constexpr int ROW_THREADS = 256;
constexpr int ZERO_BLOCKS = 64;  // blocks that clear the places in no use

// The places from `used` on, by the last ZERO_BLOCKS blocks of a grid.
template <typename T, int V>
__device__ __forceinline__ void clear_rest(T *out, long long ld, int used, long long R, int packs, int block) {
    const long long first = static_cast<long long>(min(max(used, 0), static_cast<int>(R))) * packs;
    Pack<T, V> zero;
    zero.clear();
    for (long long u = first + static_cast<long long>(block) * ROW_THREADS + threadIdx.x; u < R * packs;
         u += static_cast<long long>(ZERO_BLOCKS) * ROW_THREADS) {
        const long long r = u / packs;
        store<T, V>(out + r * ld + (u - r * packs) * V, zero);
    }
}

// A warp takes a segment of one token's row: SEG accesses per lane.  With 16-byte
// ones a single access per lane and four of the token's rows in flight serve the
// sum best (16384 tokens, 4 choices, 4096 wide in bf16: 134 us, 6.0 TB/s; two
// accesses and two rows 137, four and two 183: fewer registers, more warps); narrow
// ones want eight (5000 tokens, 6 choices, 1001 wide in FP32: 27 us, one 48).
__host__ __device__ constexpr int seg_of(int bytes) { return bytes == 16 ? 1 : bytes == 8 ? 2 : 8; }

template <typename T, int V>
__global__ void __launch_bounds__(ROW_THREADS)
gather_kernel(int T_, int J, int packs, int segments, int E, const int *__restrict__ rows,
              const int *__restrict__ offsets, const T *__restrict__ x, long long ldx, T *__restrict__ xs,
              long long ldxs, int blocks) {
    constexpr int SEG = seg_of(Pack<T, V>::BYTES);
    const long long R = static_cast<long long>(T_) * J;
    tc::grid_trigger();
    tc::grid_wait();
    if (static_cast<int>(blockIdx.x) >= blocks) {
        clear_rest<T, V>(xs, ldxs, offsets[E], R, packs, blockIdx.x - blocks);
        return;
    }
    const int unit = blockIdx.x * (ROW_THREADS / 32) + (threadIdx.x >> 5);
    const int t = unit / segments;
    if (t >= T_) return;
    const int c0 = (unit - t * segments) * SEG * 32 + (threadIdx.x & 31);
    Pack<T, V> v[SEG];
#pragma unroll
    for (int i = 0; i < SEG; ++i)
        v[i] = load_if<T, V>(c0 + 32 * i < packs, x + t * ldx + static_cast<long long>(c0 + 32 * i) * V);
    const int *at = rows + static_cast<long long>(t) * J;
    for (int j = 0; j < J; ++j) {
        const int r = at[j];
        if (r >= 0 && r < R)
#pragma unroll
            for (int i = 0; i < SEG; ++i)
                if (c0 + 32 * i < packs) store<T, V>(xs + r * ldxs + static_cast<long long>(c0 + 32 * i) * V, v[i]);
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(ROW_THREADS)
combine_kernel(int T_, int J, int packs, int segments, const int *__restrict__ rows, const float *__restrict__ weights,
               const T *__restrict__ ys, long long ldys, const T *residual, long long ldr, T *y, long long ldy) {
    constexpr int SEG = seg_of(Pack<T, V>::BYTES);
    constexpr int U = SEG <= 2 ? 4 : 2;  // rows in flight
    const long long R = static_cast<long long>(T_) * J;
    tc::grid_trigger();
    tc::grid_wait();
    const int unit = blockIdx.x * (ROW_THREADS / 32) + (threadIdx.x >> 5);
    const int t = unit / segments;
    if (t >= T_) return;
    const int c0 = (unit - t * segments) * SEG * 32 + (threadIdx.x & 31);
    const int *at = rows + static_cast<long long>(t) * J;
    const float *wt = weights + static_cast<long long>(t) * J;
    float sum[SEG][V];
#pragma unroll
    for (int i = 0; i < SEG; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) sum[i][k] = 0.0f;
    for (int j0 = 0; j0 < J; j0 += U) {
        Pack<T, V> v[U][SEG];
        float w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            w[u] = 0.0f;
            const int r = j0 + u < J ? at[j0 + u] : -1;
            const bool in = r >= 0 && r < R;
            if (in) w[u] = weights != nullptr ? wt[j0 + u] : 1.0f;
#pragma unroll
            for (int i = 0; i < SEG; ++i)
                v[u][i] = load_if<T, V>(in && c0 + 32 * i < packs, ys + r * ldys + static_cast<long long>(c0 + 32 * i) * V);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < SEG; ++i) {
                float f[V];
                v[u][i].get(f);
#pragma unroll
                for (int k = 0; k < V; ++k) sum[i][k] = fmaf(w[u], f[k], sum[i][k]);
            }
    }
#pragma unroll
    for (int i = 0; i < SEG; ++i) {
        const long long c = static_cast<long long>(c0 + 32 * i) * V;
        if (c0 + 32 * i >= packs) continue;
        if (residual != nullptr) {
            float f[V];
            load<T, V>(residual + t * ldr + c).get(f);
#pragma unroll
            for (int k = 0; k < V; ++k) sum[i][k] += f[k];
        }
        Pack<T, V> o;
        o.set(sum[i]);
        store<T, V>(y + t * ldy + c, o);
    }
}

// A warp per choice; the other choices of the token find dy in the L1 or L2.
template <typename T, int V>
__global__ void __launch_bounds__(ROW_THREADS)
combine_backward_kernel(int T_, int J, int packs, int E, const int *__restrict__ rows, const int *__restrict__ offsets,
                        const float *__restrict__ weights, const T *__restrict__ dy, long long lddy,
                        const T *__restrict__ ys, long long ldys, T *__restrict__ dys, long long lddys,
                        float *__restrict__ dweights, int blocks) {
    const long long R = static_cast<long long>(T_) * J;
    tc::grid_trigger();
    tc::grid_wait();
    if (static_cast<int>(blockIdx.x) >= blocks) {
        clear_rest<T, V>(dys, lddys, offsets[E], R, packs, blockIdx.x - blocks);
        return;
    }
    const long long i = static_cast<long long>(blockIdx.x) * (ROW_THREADS / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (i >= R) return;
    const int r = rows[i];
    if (r < 0 || r >= R) {
        if (dweights != nullptr && lane == 0) dweights[i] = 0.0f;
        return;
    }
    const float w = weights != nullptr ? weights[i] : 1.0f;
    const T *d = dy + i / J * lddy, *s = ys + r * ldys;
    T *o = dys + r * lddys;
    float dot = 0.0f;
#pragma unroll(V * sizeof(T) > 8 ? 4 : 8)
    for (int p = lane; p < packs; p += 32) {
        float g[V], f[V];
        const Pack<T, V> gv = load<T, V>(d + static_cast<long long>(p) * V);
        const Pack<T, V> fv = load_if<T, V>(dweights != nullptr, s + static_cast<long long>(p) * V);
        gv.get(g);
        fv.get(f);
#pragma unroll
        for (int k = 0; k < V; ++k) dot = fmaf(g[k], f[k], dot);
#pragma unroll
        for (int k = 0; k < V; ++k) g[k] *= w;
        Pack<T, V> q;
        q.set(g);
        store<T, V>(o + static_cast<long long>(p) * V, q);
    }
    if (dweights != nullptr) {
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, k);
        if (lane == 0) dweights[i] = dot;
    }
}

// ---- host ----------------------------------------------------------------------------
struct Span {
    uintptr_t lo = 0, hi = 0;
};
Span span(const void *p, long long rows, long long width, long long ld, long long bytes) {
    Span s;
    if (p == nullptr || rows <= 0 || width <= 0) return s;
    s.lo = reinterpret_cast<uintptr_t>(p);
    s.hi = s.lo + static_cast<uintptr_t>(((rows - 1) * ld + width) * bytes);
    return s;
}
bool overlap(const Span &a, const Span &b) { return a.lo < b.hi && b.lo < a.hi; }
bool misaligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

int check_sizes(int type, int T, int J, int H, long long E) {
    if (type < LINEAR_F32 || type > LINEAR_F16) return SGEMM_ERR_INVALID_ARG;
    if (T < 0 || J < 0 || H < 0 || E < 0 || E > LINEAR_MAX_EXPERTS || J > EXPERTS_MAX_CHOICES ||
        static_cast<long long>(T) * J > INT_MAX)
        return SGEMM_ERR_INVALID_DIM;
    return SGEMM_OK;
}
// The widest access (16, 8, 4 or 2 bytes) that rows of this address and stride allow.
int width_of(const void *p, long long ld, int type) {
    if (p == nullptr) return 16;
    const unsigned long long bits = reinterpret_cast<uintptr_t>(p) | static_cast<unsigned long long>(ld) * lt::type_bytes(type) | 16;
    return static_cast<int>(bits & (0 - bits));
}
int narrower(int a, int b) { return a < b ? a : b; }
int launched(cudaError_t err) {
    if (err == cudaSuccess) return SGEMM_OK;
    (void)cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
}
// f(element, values per access) for the type and the bytes of an access.
template <typename F>
int with_rows(int type, int bytes, F &&f) {
    if (type == LINEAR_F32)
        return bytes == 16 ? f(float(), lt::Int<4>{}) : bytes == 8 ? f(float(), lt::Int<2>{}) : f(float(), lt::Int<1>{});
    auto half = [&](auto el) {
        return bytes == 16  ? f(el, lt::Int<8>{})
               : bytes == 8 ? f(el, lt::Int<4>{})
               : bytes == 4 ? f(el, lt::Int<2>{})
                            : f(el, lt::Int<1>{});
    };
    return type == LINEAR_BF16 ? half(__nv_bfloat16()) : half(__half());
}
int segments_of(int packs, int bytes) {
    const int seg = 32 * seg_of(bytes);
    return packs / seg + (packs % seg != 0);
}
long long blocks_for(long long warps) { return (warps + ROW_THREADS / 32 - 1) / (ROW_THREADS / 32); }

template <typename I>
int sort(long long R, int E, const I *choices, int *rows, int *offsets, int *counts, cudaStream_t stream) {
    const SortPlan s = sort_plan(R, E);
    if (s.smem > 48 * 1024 &&
        (cudaFuncSetAttribute(sort_count_kernel<I>, cudaFuncAttributeMaxDynamicSharedMemorySize, SORT_SMEM) != cudaSuccess ||
         cudaFuncSetAttribute(sort_place_kernel<I>, cudaFuncAttributeMaxDynamicSharedMemorySize, SORT_SMEM) != cudaSuccess)) {
        (void)cudaGetLastError();
        return SGEMM_ERR_DEVICE;
    }
    sg_nvtx::Range r("experts: sort");
    cudaError_t err = cudaSuccess;
    if (s.blocks > 1)
        err = tc::launch(sort_count_kernel<I>, static_cast<unsigned>(s.blocks), dim3(SORT_THREADS), s.smem, stream, choices, R,
                         E, s.range, s.warps, counts);
    if (err == cudaSuccess)
        err = tc::launch(sort_place_kernel<I>, static_cast<unsigned>(s.blocks), dim3(SORT_THREADS), s.smem, stream, choices, R,
                         E, s.range, s.warps, s.blocks, static_cast<const int *>(counts), rows, offsets);
    return launched(err);
}

}  // namespace

extern "C" size_t expert_sort_workspace_size(int T, int J, int E) {
    if (T <= 0 || J <= 0 || E <= 0 || E > LINEAR_MAX_EXPERTS || static_cast<long long>(T) * J > INT_MAX) return 0;
    const SortPlan s = sort_plan(static_cast<long long>(T) * J, E);
    return s.blocks > 1 ? static_cast<size_t>(s.blocks) * E * sizeof(int) : 0;
}

extern "C" int expert_sort(int T, int J, int E, const void *choices, int choice_bytes, int *rows, int *offsets,
                           void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (choice_bytes != 4 && choice_bytes != 8) return SGEMM_ERR_INVALID_ARG;
    const int st = check_sizes(LINEAR_F32, T, J, 0, E);
    if (st != SGEMM_OK) return st;
    if (E < 1) return SGEMM_ERR_INVALID_DIM;
    const long long R = static_cast<long long>(T) * J;
    const size_t need = expert_sort_workspace_size(T, J, E);
    if (offsets == nullptr || (R > 0 && (choices == nullptr || rows == nullptr)) || (need > 0 && workspace == nullptr))
        return SGEMM_ERR_NULL_PTR;
    if (misaligned(choices, choice_bytes) || misaligned(rows, 4) || misaligned(offsets, 4) || misaligned(workspace, 16) ||
        workspace_bytes < need)
        return SGEMM_ERR_INVALID_ARG;
    const Span sc = span(choices, 1, R, R, choice_bytes), sr = span(rows, 1, R, R, 4), so = span(offsets, 1, E + 1, 1, 4),
               sw = span(workspace, 1, static_cast<long long>(need), 1, 1);
    if (overlap(sr, sc) || overlap(so, sc) || overlap(sw, sc) || overlap(sr, so) || overlap(sr, sw) || overlap(so, sw))
        return SGEMM_ERR_ALIAS;
    int *counts = static_cast<int *>(workspace);
    return choice_bytes == 4 ? sort(R, E, static_cast<const int *>(choices), rows, offsets, counts, stream)
                             : sort(R, E, static_cast<const long long *>(choices), rows, offsets, counts, stream);
}

extern "C" int expert_gather(int type, int T, int J, int H, int E, const int *rows, const int *offsets, const void *x,
                             int64_t ldx, void *xs, int64_t ldxs, cudaStream_t stream) {
    const int st = check_sizes(type, T, J, H, E);
    if (st != SGEMM_OK) return st;
    const int least = H > 1 ? H : 1, b = lt::type_bytes(type);
    if (ldx < least || ldxs < least) return SGEMM_ERR_INVALID_LD;
    const long long R = static_cast<long long>(T) * J;
    if (R == 0 || H == 0) return SGEMM_OK;
    if (rows == nullptr || offsets == nullptr || x == nullptr || xs == nullptr) return SGEMM_ERR_NULL_PTR;
    if (misaligned(rows, 4) || misaligned(offsets, 4) || misaligned(x, b) || misaligned(xs, b)) return SGEMM_ERR_INVALID_ARG;
    const Span so = span(xs, R, H, ldxs, b);
    if (overlap(so, span(x, T, H, ldx, b)) || overlap(so, span(rows, 1, R, R, 4)) || overlap(so, span(offsets, 1, E + 1, 1, 4)))
        return SGEMM_ERR_ALIAS;
    const int width = narrower(narrower(width_of(x, ldx, type), width_of(xs, ldxs, type)), width_of(x, H, type));
    const int packs = H / (width / b), segments = segments_of(packs, width);
    const long long blocks = blocks_for(static_cast<long long>(T) * segments);
    if (static_cast<long long>(T) * segments > INT_MAX - ROW_THREADS) return SGEMM_ERR_INVALID_DIM;
    sg_nvtx::Range r("experts: gather");
    return with_rows(type, width, [&](auto el, auto v) {
        using El = decltype(el);
        return launched(tc::launch(gather_kernel<El, decltype(v)::value>, static_cast<unsigned>(blocks + ZERO_BLOCKS), dim3(ROW_THREADS), 0, stream,
            T, J, packs, segments, E, rows, offsets, static_cast<const El *>(x), ldx, static_cast<El *>(xs), ldxs, static_cast<int>(blocks)));
    });
}

extern "C" int expert_combine(int type, int T, int J, int H, const int *rows, const float *weights, const void *ys,
                              int64_t ldys, const void *residual, int64_t ldr, void *y, int64_t ldy, cudaStream_t stream) {
    const int st = check_sizes(type, T, J, H, 0);
    if (st != SGEMM_OK) return st;
    const int least = H > 1 ? H : 1, b = lt::type_bytes(type);
    if (ldys < least || ldy < least || (residual != nullptr && ldr < least)) return SGEMM_ERR_INVALID_LD;
    if (T == 0 || H == 0) return SGEMM_OK;
    const long long R = static_cast<long long>(T) * J;
    if (y == nullptr || (J > 0 && (rows == nullptr || ys == nullptr))) return SGEMM_ERR_NULL_PTR;
    if (misaligned(rows, 4) || misaligned(weights, 4) || misaligned(ys, b) || misaligned(residual, b) || misaligned(y, b))
        return SGEMM_ERR_INVALID_ARG;
    const Span so = span(y, T, H, ldy, b);
    const bool in_place = residual == y && ldr == ldy;
    if (overlap(so, span(ys, R, H, ldys, b)) || overlap(so, span(rows, 1, R, R, 4)) || overlap(so, span(weights, 1, R, R, 4)) ||
        (!in_place && overlap(so, span(residual, T, H, ldr, b))))
        return SGEMM_ERR_ALIAS;
    const int width = narrower(narrower(width_of(ys, ldys, type), width_of(residual, ldr, type)),
                            narrower(width_of(y, ldy, type), width_of(y, H, type)));
    const int packs = H / (width / b), segments = segments_of(packs, width);
    const long long blocks = blocks_for(static_cast<long long>(T) * segments);
    if (static_cast<long long>(T) * segments > INT_MAX - ROW_THREADS) return SGEMM_ERR_INVALID_DIM;
    sg_nvtx::Range r("experts: combine");
    return with_rows(type, width, [&](auto el, auto v) {
        using El = decltype(el);
        return launched(tc::launch(combine_kernel<El, decltype(v)::value>, static_cast<unsigned>(blocks), dim3(ROW_THREADS), 0, stream,
            T, J, packs, segments, rows, weights, static_cast<const El *>(ys), ldys, static_cast<const El *>(residual), ldr,
            static_cast<El *>(y), ldy));
    });
}

extern "C" int expert_combine_backward(int type, int T, int J, int H, int E, const int *rows, const int *offsets,
                                       const float *weights, const void *dy, int64_t lddy, const void *ys, int64_t ldys,
                                       void *dys, int64_t lddys, float *dweights, cudaStream_t stream) {
    const int st = check_sizes(type, T, J, H, E);
    if (st != SGEMM_OK) return st;
    const int least = H > 1 ? H : 1, b = lt::type_bytes(type);
    if (lddy < least || lddys < least || (dweights != nullptr && ldys < least)) return SGEMM_ERR_INVALID_LD;
    const long long R = static_cast<long long>(T) * J;
    if (R == 0) return SGEMM_OK;
    if (rows == nullptr || offsets == nullptr || (H > 0 && (dy == nullptr || dys == nullptr || (dweights != nullptr && ys == nullptr))))
        return SGEMM_ERR_NULL_PTR;
    if (misaligned(rows, 4) || misaligned(offsets, 4) || misaligned(weights, 4) || misaligned(dy, b) || misaligned(ys, b) ||
        misaligned(dys, b) || misaligned(dweights, 4))
        return SGEMM_ERR_INVALID_ARG;
    const Span out[2] = {span(dys, R, H, lddys, b), span(dweights, 1, R, R, 4)};
    const Span in[5] = {span(dy, T, H, lddy, b), dweights != nullptr ? span(ys, R, H, ldys, b) : Span(),
                        span(rows, 1, R, R, 4), span(offsets, 1, E + 1, 1, 4), span(weights, 1, R, R, 4)};
    for (const Span &o : out)
        for (const Span &i : in)
            if (overlap(o, i)) return SGEMM_ERR_ALIAS;
    if (overlap(out[0], out[1])) return SGEMM_ERR_ALIAS;
    const int width = narrower(narrower(width_of(dy, lddy, type), dweights == nullptr ? 16 : width_of(ys, ldys, type)),
                            narrower(width_of(dys, lddys, type), width_of(dy, H, type)));
    const int packs = H / (width / b);
    const long long blocks = blocks_for(R);
    if (blocks + ZERO_BLOCKS > INT_MAX) return SGEMM_ERR_INVALID_DIM;
    sg_nvtx::Range r("experts: combine backward");
    return with_rows(type, width, [&](auto el, auto v) {
        using El = decltype(el);
        return launched(tc::launch(combine_backward_kernel<El, decltype(v)::value>, static_cast<unsigned>(blocks + ZERO_BLOCKS), dim3(ROW_THREADS), 0, stream,
            T, J, packs, E, rows, offsets, weights, static_cast<const El *>(dy), lddy, static_cast<const El *>(ys), ldys,
            static_cast<El *>(dys), lddys, dweights, static_cast<int>(blocks)));
    });
}
