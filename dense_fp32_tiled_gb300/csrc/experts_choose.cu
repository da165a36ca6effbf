// experts_choose.cu -- a router's choice of each token's experts, and its
// gradient (C ABI: include/experts.h).
//
// A warp takes a token; lane l holds the logits of experts l * NV to l * NV + NV - 1
// (in wide accesses where the rows allow them; a group of experts is then some
// lanes in a row).  The J + 1 lanes with the largest best value give a bound that
// all picks reach; the some ten experts that do are brought together, one a
// lane, and each counts those before it: its place.  (Picking one after the
// other took 36 us for 16384 tokens of 256 experts in 8 groups; this 23.)  Values are compared as
// whole numbers of the same order as the floats (0: not to be chosen), so a
// maximum over a warp is one instruction.  Bound by instructions.
//
// What is compared.  Scores are increasing in the logits, so without a bias the
// logits themselves are: no rounding enters.  With a bias (and for the sums of a
// group's best two) the order is that of the scores in 64 bits.  A warp computes
// them in 32, by the hardware's exponential and reciprocal, with a known bound on
// the error, and where two values that have to be told apart are closer than
// that, the few that matter once more in 64: for about a token in a thousand.  (All
// of them in 64 bits: 4 million exponentials at GB300's FP64 rate would take 0.3 ms.)
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "experts.h"
#include "linear_types.cuh"
#include "nvtx_range.cuh"
#include "rows.cuh"
#include "tensor_core.cuh"

namespace {

using namespace rows;

constexpr int CHOOSE_WARPS = 4;
constexpr unsigned ALL = 0xffffffffu;

struct Choose {
    const void *logits;
    long long ld;
    const float *bias;
    int *chosen;
    float *weights;
    int T, E, J, scoring, groups, kept, top, size;  // size: experts of a group
    unsigned per;                                   // e * per >> 20 = e / size
    int lanes;                                      // that hold a group, if a power of two of them do; else 0
    bool wide, wide_bias;                           // rows that allow the widest accesses
    int renormalize;
    float scale;
};

// Floats as unsigned numbers of the same order; -0 is taken for 0.
__device__ __forceinline__ uint32_t rank_of(float v) {
    const int u = __float_as_int(v + 0.0f);
    return static_cast<uint32_t>(u ^ (u >> 31 | INT_MIN));
}
__device__ __forceinline__ float of_rank(uint32_t r) { return __uint_as_float(r >> 31 ? r & 0x7fffffffu : ~r); }
__device__ __forceinline__ unsigned long long rank_of(double v) {
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(v + 0.0));
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double of_rank(unsigned long long r) {
    return __longlong_as_double(static_cast<long long>(r >> 63 ? r & 0x7fffffffffffffffull : ~r));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(ALL, v); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
        const unsigned long long o = __shfl_xor_sync(ALL, v, k);
        v = o > v ? o : v;
    }
    return v;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) v += __shfl_xor_sync(ALL, v, k);
    return v;
}
// The larger, or a NaN if either is one.
__device__ __forceinline__ float max_or_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float warp_max_f(float v) {
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) v = max_or_nan(v, __shfl_xor_sync(ALL, v, k));
    return v;
}
// logistic(l), small ones included
__device__ __forceinline__ float sigmoid(float l) {
    const float e = expf(-fabsf(l)), s = lt::fast_reciprocal(1.0f + e);
    return l < 0.0f ? e * s : s;
}
// The same for a comparison: see `slack`.
__device__ __forceinline__ float sigmoid_about(float l) { return lt::fast_reciprocal(1.0f + lt::fast_exp2(-lt::kLog2E * l)); }

// A lane's NV values of a row of E, outside for those that the row has not.
template <typename T, int NV>
__device__ __forceinline__ void load_row(const T *row, int lane, int E, bool wide, float outside, float (&f)[NV]) {
    constexpr int BYTES = NV * static_cast<int>(sizeof(T)) < 16 ? NV * static_cast<int>(sizeof(T)) : 16;
    constexpr int N = BYTES / static_cast<int>(sizeof(T));
    if (wide) {
        Pack<T, N> p[NV / N];
#pragma unroll
        for (int a = 0; a < NV / N; ++a) p[a] = load_if<T, N>(lane * NV + a * N < E, row + lane * NV + a * N);
#pragma unroll
        for (int a = 0; a < NV / N; ++a) {
            float v[N];
            p[a].get(v);
#pragma unroll
            for (int k = 0; k < N; ++k) f[a * N + k] = lane * NV + a * N < E ? v[k] : outside;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) f[i] = lane * NV + i < E ? to_f(row[lane * NV + i]) : outside;
    }
}

template <typename T, int NV>
__device__ __forceinline__ void store_row(T *row, int lane, int E, bool wide, const float (&f)[NV]) {
    constexpr int BYTES = NV * static_cast<int>(sizeof(T)) < 16 ? NV * static_cast<int>(sizeof(T)) : 16;
    constexpr int N = BYTES / static_cast<int>(sizeof(T));
    if (wide) {
#pragma unroll
        for (int a = 0; a < NV / N; ++a) {
            float v[N];
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = f[a * N + k];
            Pack<T, N> p;
            p.set(v);
            if (lane * NV + a * N < E) store<T, N>(row + lane * NV + a * N, p);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane * NV + i < E) row[lane * NV + i] = from_f<T>(f[i]);
    }
}

// The sum of the two largest of a warp's values (ranks; each lane gives its own best two; 0: none).
template <typename R, typename F>
__device__ __forceinline__ F best_two(R first, R second, bool two, R *any) {
    const R high = warp_max(first);
    *any = high;
    if (high == 0) return 0;
    F sum = of_rank(high);
    if (two) {
        const int owner = __ffs(__ballot_sync(ALL, first == high)) - 1;
        const R next = warp_max(static_cast<int>(threadIdx.x & 31) == owner ? second : first);
        if (next != 0) sum += of_rank(next);
    }
    return sum;
}
template <typename R>
__device__ __forceinline__ void keep_two(R r, R &first, R &second) {
    second = r > first ? first : r > second ? r : second;
    first = r > first ? r : first;
}
__device__ __forceinline__ unsigned group_of(const Choose &c, int e) { return e * c.per >> 20; }

// A token's scores for comparing: m its largest logit, most = 1 / sum of exp(l - m).
struct Scores {
    bool softmax;
    float m, most;
    __device__ __forceinline__ float of(float l) const { return softmax ? expf(l - m) * most : sigmoid_about(l); }
    __device__ __forceinline__ float with(float l, float bias) const { return __fadd_rn(of(l), bias); }  // the same bits everywhere
};

// ---- in 64 bits: for few tokens, so in little code (an SM fetches it anew) -----------
// A warp's room: the experts whose values are told apart, in order, and their ranks.
struct Held {
    unsigned long long *rank;
    unsigned short *expert;
};
// Brings together the experts of the groups in `mask` whose values in 32 bits are not
// below `least` (lane g's: of group g) and works out their values.  How many there are.
// (All in one pass of the exponential and the quotient, which take a warp 2 us.)
template <typename T>
__device__ __noinline__ int values_in_64(const Choose &c, const T *row, const Held &held, const Scores &s, unsigned mask, float least,
                                         int lane) {
    int n = 0;
#pragma unroll 1
    for (int first = 0; first < c.E; first += 32) {
        const int e = first + lane;
        const unsigned g = e < c.E ? group_of(c, e) : 0;
        const float bound = __shfl_sync(ALL, least, g);
        bool in = false;
        if (e < c.E && (mask >> g & 1) != 0) {
            const float l = to_f(row[e]), b = c.bias != nullptr ? c.bias[e] : 0.0f;
            in = l > -INFINITY && b > -INFINITY && !(s.with(l, b) < bound);
        }
        const unsigned all = __ballot_sync(ALL, in);
        if (in) held.expert[n + __popc(all & ((1u << lane) - 1))] = static_cast<unsigned short>(e);
        n += __popc(all);
    }
    double z = 1.0;  // without a bias the scores' proportions are enough
    if (s.softmax && c.bias != nullptr) {
        z = 0.0;
#pragma unroll 1
        for (int e = lane; e < c.E; e += 32) z += exp(static_cast<double>(to_f(row[e])) - static_cast<double>(s.m));
        z = warp_sum(z);
    }
    __syncwarp();
#pragma unroll 1
    for (int k = lane; k < n; k += 32) {
        const int e = held.expert[k];
        // exp(l - m) / z, or 1 / (1 + exp(-l)) in the form that keeps small ones
        const double l = static_cast<double>(to_f(row[e])), x = exp(s.softmax ? l - static_cast<double>(s.m) : -fabs(l));
        const double v = (s.softmax || l < 0.0 ? x : 1.0) / (s.softmax ? z : 1.0 + x);
        held.rank[k] = rank_of(c.bias != nullptr ? v + static_cast<double>(c.bias[e]) : v);
    }
    __syncwarp();
    return n;
}
// The groups that compete, of which `keep` do by sums in 32 bits: those whose sums are
// within `width` of the border's other side (low: the least that stays, out: the
// largest that does not) by their sums in 64.
template <typename T>
__device__ __noinline__ unsigned groups_in_64(const Choose &c, const T *row, const Held &held, const Scores &s, unsigned keep,
                                              uint32_t total, uint32_t least, float low, float out, float width, int lane) {
    const float v = of_rank(total);
    const bool stays = (keep >> lane & 1) != 0;
    const unsigned near = __ballot_sync(ALL, lane < c.groups && total != 0 && !((stays ? v - out : low - v) >= width));
    // a group's best are among those not further below its last one in 32 bits: 2 scores, 2 sums with the
    // bias, and what `least` lost
    const int n = values_in_64(c, row, held, s, near, least != 0 ? of_rank(least) - width : -INFINITY, lane);
    unsigned long long exact = 0;  // lane g
    int before = 0;
#pragma unroll 1
    for (unsigned left = near; left != 0; left &= left - 1) {
        const int g = __ffs(left) - 1;
        unsigned long long first = 0, second = 0, any;
        for (int k = lane; k < n; k += 32)
            if (group_of(c, held.expert[k]) == static_cast<unsigned>(g)) keep_two(held.rank[k], first, second);
        const double sum = best_two<unsigned long long, double>(first, second, c.top > 1, &any);
        if (lane == g) exact = rank_of(sum);
    }
#pragma unroll 1
    for (unsigned left = near; left != 0; left &= left - 1) {
        const int g = __ffs(left) - 1;
        const unsigned long long o = __shfl_sync(ALL, exact, g);
        before += o > exact || (o == exact && g < lane) ? 1 : 0;
    }
    return (keep & ~near) | __ballot_sync(ALL, (near >> lane & 1) != 0 && before < __popc(keep & near));
}
// The J best of the groups in `mask`, of those not below `least`: this lane's picks
// (pick j at lane j % 32, in mine[j / 32]).
template <typename T>
__device__ __noinline__ void picks_in_64(const Choose &c, const T *row, const Held &held, const Scores &s, unsigned mask, float least,
                                         int lane, int *mine) {
    const int n = values_in_64(c, row, held, s, mask, least, lane);
    mine[0] = mine[1] = -1;
    if (n <= 32) {  // each counts those before it
        const unsigned long long k = lane < n ? held.rank[lane] : 0;
        const int e = lane < n ? held.expert[lane] : -1;
        int place = 0;
#pragma unroll 1
        for (int o = 0; o < n; ++o) {
            const unsigned long long other = __shfl_sync(ALL, k, o);
            place += other > k || (other == k && o < lane) ? 1 : 0;
        }
        __syncwarp();
        if (e >= 0) held.expert[place] = static_cast<unsigned short>(e);
        __syncwarp();
        if (lane < n && lane < c.J) mine[0] = held.expert[lane];
        __syncwarp();
        return;
    }
#pragma unroll 1
    for (int j = 0; j < c.J; ++j) {
        unsigned long long best = 0;
        int at = INT_MAX;
#pragma unroll 1
        for (int k = lane; k < n; k += 32)
            if (held.rank[k] > best) {
                best = held.rank[k];
                at = k;
            }
        const unsigned long long high = warp_max(best);
        if (high == 0) break;
        const int pick = __reduce_min_sync(ALL, best == high ? at : INT_MAX);
        if ((j & 31) == lane) mine[j >> 5] = held.expert[pick];
        __syncwarp();
        if (at == pick) held.rank[at] = 0;
        __syncwarp();
    }
}

// The last pick (logit lp, bias bp, value v) and the first expert that is left out are equal, which their
// numbers decide.  Whether an expert with another logit or bias lies so near (`width`) that it may come
// before both.  The scores are worked out again: kept, they cost every token registers (16384 x 256 in 8 groups
// 24.2 us for 23.3, without groups and of logits in half numbers, where many tokens come here, 18 for 22).  A lane's own
// experts in wide accesses; where those are many, one after the other, for the kernel's registers.
template <typename T, int NV>
__device__ __noinline__ bool others_near(const Choose &c, const T *row, const Scores &s, unsigned mask, float lp, float bp, float v,
                                         float width, int lane) {
    bool near = false;
    auto look = [&](int e, float l, float b) {
        const bool in = (mask >> (group_of(c, e) & 31) & 1) != 0 && l > -INFINITY && b > -INFINITY;
        near |= in && !(fabsf(v - s.with(l, b)) >= width) && !(l == lp && b == bp);
    };
    if constexpr (NV <= 8) {
        float l[NV], b[NV];
        load_row<T, NV>(row, lane, c.E, c.wide, -INFINITY, l);
        load_row<float, NV>(c.bias, lane, c.E, c.wide_bias, -INFINITY, b);
#pragma unroll
        for (int i = 0; i < NV; ++i) look(lane * NV + i, l[i], b[i]);
    } else {
#pragma unroll 1
        for (int e = lane; e < c.E; e += 32) look(e, to_f(row[e]), c.bias[e]);
    }
    return __any_sync(ALL, near);
}

template <typename T, int NV>
__global__ void __launch_bounds__(CHOOSE_WARPS * 32, NV <= 8 ? 32 / CHOOSE_WARPS : 1) choose_kernel(const __grid_constant__ Choose c) {
    extern __shared__ unsigned long long room[];
    __shared__ int picks[CHOOSE_WARPS][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * CHOOSE_WARPS + warp;
    tc::grid_trigger();
    tc::grid_wait();
    if (t >= c.T) return;
    const T *row = static_cast<const T *>(c.logits) + t * c.ld;
    Held held;
    held.rank = room + static_cast<size_t>(warp) * c.E;
    held.expert = reinterpret_cast<unsigned short *>(room + static_cast<size_t>(CHOOSE_WARPS) * c.E) + warp * c.E;
    const int e0 = lane * NV;
    float l[NV];
    load_row<T, NV>(row, lane, c.E, c.wide, -INFINITY, l);
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) m = max_or_nan(m, l[i]);
    m = warp_max_f(m);
    Scores s{c.scoring == EXPERTS_SOFTMAX, m, 1.0f};
    if (m != m || (s.softmax && m == INFINITY)) {
        for (int j = lane; j < c.J; j += 32) {
            c.chosen[static_cast<long long>(t) * c.J + j] = -1;
            c.weights[static_cast<long long>(t) * c.J + j] = __int_as_float(0x7fffffff);
        }
        return;
    }
    const bool summed = c.groups > 1 && c.top > 1;  // groups by sums of scores
    if (s.softmax && (c.bias != nullptr || !c.renormalize || summed) && m > -INFINITY) {
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) z += expf(l[i] - m);
        s.most = lt::fast_reciprocal(warp_sum(z));
    }
    // How far the difference of two scores may be off, in units of 2^-24.  Sigmoid: the exponential is
    // within 4 of its value and the rounding of its argument moves it by 1.44 |l|, of which a quarter and
    // 0.33 at most reach the score; the sum adds 1, the reciprocal 2: 5 a score.  Softmax, of the largest
    // score 1 / z: 4 of its own exponential (expf), less than 1 of the rounding of l - m (x exp(-x) < 0.4),
    // and those of z: 36 of up to 31 sums in a lane and 5 across, 11 of the exponentials (4, and the
    // rounding of l - m at a mean of up to log 1024); 3 of reciprocal and product.
    const float slack = s.softmax ? s.most * 0x1p-17f : 0x1p-20f;
    uint32_t key[NV];
    if (c.bias != nullptr) {
        float bias[NV];
        load_row<float, NV>(c.bias, lane, c.E, c.wide_bias, -INFINITY, bias);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float v = s.with(l[i], bias[i]);
            key[i] = l[i] > -INFINITY && v > -INFINITY ? rank_of(v) : 0;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = l[i] > -INFINITY ? rank_of(l[i]) : 0;
    }
    unsigned keep = 1;  // a bit a group
    if (c.groups > 1) {
        uint32_t total = 0, least = 0;  // lane g: the rank of group g's sum, and of the least value in it
        const bool scores = summed && c.bias == nullptr;
        auto value_rank = [&](int i) { return scores && key[i] != 0 ? rank_of(s.of(l[i])) : key[i]; };
        if (c.lanes > 0) {  // a group is `lanes` lanes, a power of two
            uint32_t first = 0, second = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) keep_two(value_rank(i), first, second);
            for (int k = 1; k < c.lanes; k <<= 1) {
                const uint32_t o1 = __shfl_xor_sync(ALL, first, k), o2 = __shfl_xor_sync(ALL, second, k);
                keep_two(o1, first, second);
                keep_two(o2, first, second);
            }
            float sum = of_rank(first);
            if (c.top > 1 && second != 0) sum += of_rank(second);
            total = __shfl_sync(ALL, first != 0 ? rank_of(sum) : 0, lane * c.lanes & 31);
            least = __shfl_sync(ALL, c.top > 1 ? second : first, lane * c.lanes & 31);
            if (lane >= c.groups) total = 0;
        } else {
            for (int g = 0; g < c.groups; ++g) {
                uint32_t first = 0, second = 0, any;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (group_of(c, e0 + i) == static_cast<unsigned>(g)) keep_two(value_rank(i), first, second);
                const float sum = best_two<uint32_t, float>(first, second, c.top > 1, &any);
                const int values = __popc(__ballot_sync(ALL, first != 0)) + __popc(__ballot_sync(ALL, second != 0));
                if (lane == g && any != 0) {
                    total = rank_of(sum);
                    least = c.top == 1 ? total : values < 2 ? 0 : rank_of(sum - of_rank(any));
                }
            }
        }
        // group g's place: those before it (lanes without a group hold 0)
        int before = 0;
        for (int g = 0; g < c.groups; g += 4)
#pragma unroll
            for (int u = 0; u < 4; ++u)
                before += __shfl_sync(ALL, total, g + u & 31) > total - (g + u < lane ? 1u : 0u) ? 1 : 0;
        const bool stays = total != 0 && before < c.kept;
        keep = __ballot_sync(ALL, stays);
        if (summed || c.bias != nullptr) {
            const uint32_t low = __reduce_min_sync(ALL, stays ? total : 0xffffffffu), out = warp_max(stays ? 0u : total);
            if (out != 0) {
                const float a = of_rank(least), v = of_rank(total);  // of what the sums add up: the size
                float size = total == 0 ? 0.0f : least == 0 ? fabsf(v) : fmaxf(fabsf(a), fabsf(v - a));
#pragma unroll
                for (int k = 16; k > 0; k >>= 1) size = fmaxf(size, __shfl_xor_sync(ALL, size, k));
                const float width = 2.0f * slack + 0x1p-21f * size;  // 4 scores; 4 sums with biases, 2 of two values
                if (!(of_rank(low) - of_rank(out) >= width))
                    keep = groups_in_64(c, row, held, s, keep, total, least, of_rank(low), of_rank(out), width, lane);
            }
        }
        if (c.lanes > 0) {
            const bool in = (keep >> (group_of(c, e0) & 31) & 1) != 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) key[i] = in ? key[i] : 0;
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if ((keep >> (group_of(c, e0 + i) & 31) & 1) == 0) key[i] = 0;
        }
    }
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) best = key[i] > best ? key[i] : best;
    int mine[2] = {-1, -1}, *pick = picks[warp];
    float floor = 0.0f;  // the least pick's value
    bool doubt = false;
    int n = 33, count = 0, at_list = 0;
    uint32_t mask = 0;  // of this lane's experts, those brought together
    if (c.J < 32) {
        // of as many lanes' best as there are picks and one more, the least: a bound
        uint32_t left = best, bound;
        int need = c.J;
        do {
            bound = warp_max(left);
            need -= __popc(__ballot_sync(ALL, left == bound));
            left = left == bound ? 0 : left;
        } while (need >= 0 && bound != 0);
        bound = bound > 1 ? bound : 1;
#pragma unroll
        for (int i = 0; i < NV; ++i) mask |= key[i] >= bound ? 1u << i : 0u;
        count = __popc(mask);
        n = count;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int o = __shfl_up_sync(ALL, n, k);
            if (lane >= k) n += o;
        }
        at_list = n - count;
        n = __shfl_sync(ALL, n, 31);
    }
    if (n <= 32) {
        for (; mask != 0; mask &= mask - 1) pick[at_list++] = e0 + __ffs(mask) - 1;
        __syncwarp();
        int e = lane < n ? pick[lane] : -1;
        // its value again, as its lane has it
        float le = e >= 0 ? to_f(row[e]) : 0.0f, be = e >= 0 && c.bias != nullptr ? c.bias[e] : 0.0f;
        float v = c.bias != nullptr ? s.with(le, be) : le;
        const uint32_t k = e >= 0 ? rank_of(v) : 0;
        int place = 0;
        for (int o = 0; o < n; o += 4)  // lanes without an expert hold 0
#pragma unroll
            for (int u = 0; u < 4; ++u) place += __shfl_sync(ALL, k, o + u & 31) > k - (o + u < lane ? 1u : 0u) ? 1 : 0;
        __syncwarp();
        if (e >= 0) pick[place] = lane;
        __syncwarp();
        const int from = lane < n ? pick[lane] : 0;
        e = __shfl_sync(ALL, e, from);
        if (lane < c.J && lane < n) mine[0] = e;
        if (c.bias != nullptr) {
            // neighbours among the picks and the first that is none: 2 scores, 2 sums with the bias; values of equal
            // logits and biases are equal in 64 bits too
            v = __shfl_sync(ALL, v, from);
            floor = __shfl_sync(ALL, v, min(c.J, n) - 1 & 31);
            const float next = __shfl_down_sync(ALL, v, 1);
            const bool close = lane < c.J && lane + 1 < n && !(v - next >= slack + 0x1p-22f * fabsf(v));
            if (__any_sync(ALL, close)) {
                le = __shfl_sync(ALL, le, from);
                be = __shfl_sync(ALL, be, from);
                const float ln = __shfl_down_sync(ALL, le, 1), bn = __shfl_down_sync(ALL, be, 1);
                const unsigned equal = __ballot_sync(ALL, close && le == ln && be == bn);
                doubt = __ballot_sync(ALL, close) != equal;
                if (!doubt && c.J < n && (equal >> (c.J - 1) & 1) != 0)  // what is behind both may come before them
                    doubt = others_near<T, NV>(c, row, s, keep, __shfl_sync(ALL, le, c.J - 1), __shfl_sync(ALL, be, c.J - 1), floor,
                                        slack + 0x1p-22f * fabsf(floor), lane);
            }
        }
    } else {  // many picks or many equal values: one after the other
        uint32_t taken = 0;
        int at = INT_MAX;
        auto look = [&] {
            best = 0;
            at = INT_MAX;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if ((taken >> i & 1) == 0 && key[i] > best) {
                    best = key[i];
                    at = e0 + i;
                }
        };
        look();
        float last = 0.0f;
        int last_who = -1;
        const int rounds = c.bias != nullptr ? c.J + 1 : c.J;  // one more: the best that is left out
        for (int j = 0; j < rounds; ++j) {
            const uint32_t high = warp_max(best);
            if (high == 0) break;
            const int who = __reduce_min_sync(ALL, best == high ? at : INT_MAX);
            if (c.bias != nullptr) {
                const float v = of_rank(high);
                if (j > 0 && !doubt && !(last - v >= slack + 0x1p-22f * fabsf(last))) {
                    const float l_last = to_f(row[last_who]), b_last = c.bias[last_who];
                    doubt = !(to_f(row[who]) == l_last && c.bias[who] == b_last);
                    if (!doubt && j == c.J) doubt = others_near<T, NV>(c, row, s, keep, l_last, b_last, last, slack + 0x1p-22f * fabsf(last), lane);
                }
                last = v;
                last_who = who;
                if (j < c.J) floor = v;
            }
            if (j < c.J && (j & 31) == lane) mine[j >> 5] = who;
            if (who == at) {
                taken |= 1u << (who - e0);
                look();
            }
        }
    }
    if (doubt)  // those that may be among the J best, in 64 bits
        picks_in_64(c, row, held, s, keep, floor - slack - 0x1p-22f * fabsf(floor), lane, mine);

    // weights of the picks
    float lj[2], w[2];
    float high = -INFINITY;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        lj[u] = mine[u] >= 0 ? to_f(row[mine[u]]) : -INFINITY;
        high = fmaxf(high, lj[u]);
    }
    float sum = 0.0f;
    const int slots = c.J > 32 ? 2 : 1;
    if (c.renormalize) {
        // relative to the largest pick, so that no pick's score is lost below the smallest number
        high = warp_max_f(high);
        const float ref = s.softmax ? high : fminf(high, 0.0f);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (u >= slots) break;
            w[u] = s.softmax || lj[u] < 0.0f ? expf(lj[u] - ref) : 1.0f;
            if (!s.softmax) w[u] *= lt::fast_reciprocal(1.0f + expf(-fabsf(lj[u])));
            if (mine[u] < 0) w[u] = 0.0f;
            sum += w[u];
        }
        sum = warp_sum(sum);
    }
    const float share = lt::fast_reciprocal(sum);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        if (u >= slots) break;
        if (c.renormalize)
            w[u] *= share;
        else
            w[u] = s.softmax ? expf(lj[u] - m) * s.most : sigmoid(lj[u]);
        w[u] = mine[u] < 0 ? 0.0f : w[u] * c.scale;
        const int j = u * 32 + lane;
        if (j < c.J) {
            c.chosen[static_cast<long long>(t) * c.J + j] = mine[u];
            c.weights[static_cast<long long>(t) * c.J + j] = w[u];
        }
    }
}

// ---- gradient -----------------------------------------------------------------------
struct ChooseBackward {
    const float *dweights;
    const int *chosen;
    const void *logits;
    void *dlogits;
    long long ld, ldd;
    int T, E, J, scoring, renormalize;
    bool wide;  // rows that allow the widest accesses
    float scale;
};

// A warp takes a token: lane j works out the gradient of pick j (and of j + 32),
// then each lane gathers those of its experts, in the order of the picks.
template <typename T, int NV>
__global__ void __launch_bounds__(CHOOSE_WARPS * 32) choose_backward_kernel(const __grid_constant__ ChooseBackward c) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * CHOOSE_WARPS + (threadIdx.x >> 5);
    tc::grid_trigger();
    tc::grid_wait();
    if (t >= c.T) return;
    const T *row = static_cast<const T *>(c.logits) + t * c.ld;
    const bool softmax = c.scoring == EXPERTS_SOFTMAX, all = softmax && !c.renormalize;
    int e[2];
    float l[2], p[2], g[2];
    float high = -INFINITY;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int j = s * 32 + lane;
        const long long at = static_cast<long long>(t) * c.J + j;
        e[s] = j < c.J ? c.chosen[at] : -1;
        if (e[s] < 0 || e[s] >= c.E) e[s] = -1;
        g[s] = e[s] >= 0 ? c.dweights[at] * c.scale : 0.0f;
        l[s] = e[s] >= 0 ? to_f(row[e[s]]) : -INFINITY;
        high = fmaxf(high, l[s]);
    }
    const bool any = __any_sync(ALL, e[0] >= 0 || e[1] >= 0);
    float x[NV];
    float z = 1.0f;
    if (all) {
        high = -INFINITY;
        load_row<T, NV>(row, lane, c.E, c.wide, -INFINITY, x);
#pragma unroll
        for (int i = 0; i < NV; ++i) high = fmaxf(high, x[i]);
        high = warp_max_f(high);
        z = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i] = expf(x[i] - high);
            z += x[i];
        }
        z = warp_sum(z);
    } else {
        high = warp_max_f(high);
    }
    // the picks' shares of what they are divided by, and with those the mean of the weights' gradients
    const float ref = softmax ? high : fminf(high, 0.0f);
    float sum = 0.0f;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        p[s] = softmax || l[s] < 0.0f ? expf(l[s] - ref) : 1.0f;
        if (!softmax) p[s] *= lt::fast_reciprocal(1.0f + expf(-fabsf(l[s])));
        if (e[s] < 0) p[s] = 0.0f;
        sum += p[s];
    }
    const float whole = all ? z : warp_sum(sum);
    const float share = any ? lt::fast_reciprocal(whole) : 1.0f;
    float mean = 0.0f;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        p[s] *= share;
        mean += p[s] * g[s];
    }
    mean = softmax || c.renormalize ? warp_sum(mean) : 0.0f;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const float far = sigmoid(-l[s]);  // 1 - sigmoid(l)
        if (all)
            ;  // joined with the other experts below
        else if (softmax)
            g[s] = p[s] * (g[s] - mean);
        else if (c.renormalize)
            g[s] = p[s] * far * (g[s] - mean);
        else
            g[s] *= sigmoid(l[s]) * far;
        if (e[s] < 0) g[s] = 0.0f;
    }
    float d[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) d[i] = 0.0f;
    for (int j = 0; j < c.J; ++j) {
        const int who = __shfl_sync(ALL, j < 32 ? e[0] : e[1], j & 31);
        const float what = __shfl_sync(ALL, j < 32 ? g[0] : g[1], j & 31);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane * NV + i == who) d[i] += what;
    }
    T *out = static_cast<T *>(c.dlogits) + t * c.ldd;
    if (all) {
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] = any ? x[i] * share * (d[i] - mean) : 0.0f;
    }
    store_row<T, NV>(out, lane, c.E, c.wide, d);
}

// ---- host ----------------------------------------------------------------------------
// f(values per lane) for E experts.
template <typename F>
int with_experts(int E, F &&f) {
    return E <= 32    ? f(lt::Int<1>{})
           : E <= 64  ? f(lt::Int<2>{})
           : E <= 128 ? f(lt::Int<4>{})
           : E <= 256 ? f(lt::Int<8>{})
           : E <= 512 ? f(lt::Int<16>{})
                      : f(lt::Int<32>{});
}
// Whether rows of E values allow load_row's accesses with nv values a lane.
bool wide_rows(const void *p, long long ld, int E, int bytes, int nv) {
    const int access = nv * bytes < 16 ? nv * bytes : 16;
    return reinterpret_cast<uintptr_t>(p) % access == 0 && ld * bytes % access == 0 && static_cast<long long>(E) * bytes % access == 0;
}
int check_choice(int type, int T, int E, int J, int scoring) {
    if (type < LINEAR_F32 || type > LINEAR_F16 || (scoring != EXPERTS_SOFTMAX && scoring != EXPERTS_SIGMOID))
        return SGEMM_ERR_INVALID_ARG;
    if (T < 0 || E < 1 || E > EXPERTS_MAX_CHOOSE || J < 0 || J > E || J > EXPERTS_MAX_CHOICES ||
        T > INT_MAX - CHOOSE_WARPS || static_cast<long long>(T) * J > INT_MAX)
        return SGEMM_ERR_INVALID_DIM;
    return SGEMM_OK;
}
unsigned token_blocks(int T) { return static_cast<unsigned>((T + CHOOSE_WARPS - 1) / CHOOSE_WARPS); }

}  // namespace

extern "C" int expert_choose(int type, int T, int E, int J, const void *logits, int64_t ldl, const float *bias, int scoring,
                             int groups, int kept_groups, int group_top, int renormalize, float scale, int *chosen,
                             float *weights, cudaStream_t stream) {
    int st = check_choice(type, T, E, J, scoring);
    if (st != SGEMM_OK) return st;
    if (groups < 1 || groups > EXPERTS_MAX_GROUPS || E % groups != 0 || kept_groups < 1 || kept_groups > groups ||
        (group_top != 1 && group_top != 2))
        return SGEMM_ERR_INVALID_ARG;
    if (ldl < E) return SGEMM_ERR_INVALID_LD;
    if (T == 0 || J == 0) return SGEMM_OK;
    if (logits == nullptr || chosen == nullptr || weights == nullptr) return SGEMM_ERR_NULL_PTR;
    const int b = lt::type_bytes(type);
    if (misaligned(logits, b) || misaligned(bias, 4) || misaligned(chosen, 4) || misaligned(weights, 4))
        return SGEMM_ERR_INVALID_ARG;
    const long long R = static_cast<long long>(T) * J;
    const Span sl = span(logits, T, E, ldl, b), sb = span(bias, 1, E, E, 4), sc = span(chosen, 1, R, R, 4),
               sw = span(weights, 1, R, R, 4);
    if (overlap(sc, sl) || overlap(sc, sb) || overlap(sw, sl) || overlap(sw, sb) || overlap(sc, sw)) return SGEMM_ERR_ALIAS;
    Choose c{};
    c.logits = logits, c.ld = ldl, c.bias = bias, c.chosen = chosen, c.weights = weights, c.T = T, c.E = E, c.J = J;
    c.scoring = scoring, c.groups = groups, c.kept = kept_groups, c.top = group_top, c.size = E / groups;
    c.per = (1u << 20) / static_cast<unsigned>(c.size) + 1;  // exact for e * size < 2^20
    c.renormalize = renormalize != 0, c.scale = scale;
    if (groups == 1) c.top = 1;
    const bool in_64 = bias != nullptr || (groups > 1 && group_top > 1);
    const size_t smem = in_64 ? (sizeof(unsigned long long) + sizeof(unsigned short)) * CHOOSE_WARPS * static_cast<size_t>(E) : 0;
    sg_nvtx::Range r("experts: choose");
    return with_experts(E, [&](auto n) {
        constexpr int NV = decltype(n)::value;
        c.wide = wide_rows(logits, ldl, E, b, NV);
        c.wide_bias = wide_rows(bias, 0, E, 4, NV);
        const int lanes = c.size / NV;
        c.lanes = c.size % NV == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
        auto run = [&](auto kernel) { return launched(tc::launch(kernel, token_blocks(T), dim3(CHOOSE_WARPS * 32), smem, stream, c)); };
        return type == LINEAR_F32    ? run(choose_kernel<float, NV>)
               : type == LINEAR_BF16 ? run(choose_kernel<__nv_bfloat16, NV>)
                                     : run(choose_kernel<__half, NV>);
    });
}

extern "C" int expert_choose_backward(int type, int T, int E, int J, const float *dweights, const int *chosen,
                                      const void *logits, int64_t ldl, int scoring, int renormalize, float scale,
                                      void *dlogits, int64_t ldd, cudaStream_t stream) {
    int st = check_choice(type, T, E, J, scoring);
    if (st != SGEMM_OK) return st;
    if (ldl < E || ldd < E) return SGEMM_ERR_INVALID_LD;
    if (T == 0) return SGEMM_OK;
    if (logits == nullptr || dlogits == nullptr || (J > 0 && (chosen == nullptr || dweights == nullptr))) return SGEMM_ERR_NULL_PTR;
    const int b = lt::type_bytes(type);
    if (misaligned(logits, b) || misaligned(dlogits, b) || misaligned(chosen, 4) || misaligned(dweights, 4))
        return SGEMM_ERR_INVALID_ARG;
    const long long R = static_cast<long long>(T) * J;
    const Span so = span(dlogits, T, E, ldd, b);
    if (overlap(so, span(logits, T, E, ldl, b)) || overlap(so, span(chosen, 1, R, R, 4)) || overlap(so, span(dweights, 1, R, R, 4)))
        return SGEMM_ERR_ALIAS;
    ChooseBackward c{};
    c.dweights = dweights, c.chosen = chosen, c.logits = logits, c.dlogits = dlogits, c.ld = ldl, c.ldd = ldd;
    c.T = T, c.E = E, c.J = J, c.scoring = scoring, c.renormalize = renormalize != 0, c.scale = scale;
    sg_nvtx::Range r("experts: choose backward");
    return with_experts(E, [&](auto n) {
        constexpr int NV = decltype(n)::value;
        c.wide = wide_rows(logits, ldl, E, b, NV) && wide_rows(dlogits, ldd, E, b, NV);
        auto run = [&](auto kernel) { return launched(tc::launch(kernel, token_blocks(T), dim3(CHOOSE_WARPS * 32), 0, stream, c)); };
        return type == LINEAR_F32    ? run(choose_backward_kernel<float, NV>)
               : type == LINEAR_BF16 ? run(choose_backward_kernel<__nv_bfloat16, NV>)
                                     : run(choose_backward_kernel<__half, NV>);
    });
}
