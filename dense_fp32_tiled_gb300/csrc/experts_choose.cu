// experts_choose.cu -- a router's choice of each token's experts, and its
// gradient (C ABI: include/experts.h).
//
// A warp takes a token; lane l holds the logits of experts l * NV to l * NV + NV - 1
// (in wide accesses where the rows allow them; a group of experts is then some
// lanes in a row).  The J + 1 lanes with the largest best value give a bound that
// all picks reach; the some ten experts that do are brought together, one a
// lane, and each counts those before it: its place.  (Picking one after the
// other took 36 us for 16384 tokens of 256 experts in 8 groups; this NN.)  Values are compared as
// whole numbers of the same order as the floats (0: not to be chosen), so a
// maximum over a warp is one instruction.  Bound by instructions.
//
// What is compared.  Scores are increasing in the logits, so without a bias the
// logits themselves are: no rounding enters.  With a bias (and for the sums of a
// group's best two) the order is that of the scores in 64 bits.  A warp computes
// them in 32, by the hardware's exponential and reciprocal, with a known bound on
// the error, and where two values that have to be told apart are closer than
// that, the few that matter once more in 64: for some tokens in a hundred.  (All
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
__device__ __forceinline__ double sigmoid(double l) {
    const double e = exp(-fabs(l));
    return l < 0.0 ? e / (1.0 + e) : 1.0 / (1.0 + e);
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
// Which groups compete, a bit each: lane g holds the rank of group g's sum (0: none of its experts may be chosen).
__device__ __forceinline__ unsigned kept_groups(const Choose &c, uint32_t total, int lane) {
    unsigned keep = 0;
    for (int k = 0; k < c.kept; ++k) {
        const uint32_t high = warp_max(total);
        if (high == 0) break;
        const unsigned one = __ballot_sync(ALL, total == high);
        keep |= one & (0u - one);  // the lowest
        if ((keep >> lane & 1) != 0) total = 0;
    }
    return keep;
}
__device__ __forceinline__ unsigned group_of(const Choose &c, int e) { return e * c.per >> 20; }

// A warp's room: ranks and numbers of experts whose values are told apart in 64 bits.
struct Held {
    unsigned long long *rank;
    unsigned short *expert;
};

// Puts the experts of this lane for which which(i) holds into `held`, all lanes' in
// the order of their numbers.  How many there are; none are put there if more than `room`.
template <int NV, typename I, typename F>
__device__ __forceinline__ int bring_together(I *expert, int room, int e0, int lane, F &&which) {
    int mine = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) mine += which(i) ? 1 : 0;
    int n = mine;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const int o = __shfl_up_sync(ALL, n, k);
        if (lane >= k) n += o;
    }
    int at = n - mine;
    n = __shfl_sync(ALL, n, 31);
    __syncwarp();
    if (n <= room) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (which(i)) expert[at++] = static_cast<I>(e0 + i);
    }
    __syncwarp();
    return n;
}

// The values of the n experts of `held` in 64 bits.
template <typename T>
__device__ __noinline__ void values_in_64(const Choose &c, const T *row, const Held &held, int n, int lane) {
    double m = -INFINITY, z = 0.0;
    if (c.scoring == EXPERTS_SOFTMAX) {
        for (int e = lane; e < c.E; e += 32) m = fmax(m, static_cast<double>(to_f(row[e])));
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) m = fmax(m, __shfl_xor_sync(ALL, m, k));
        for (int e = lane; e < c.E; e += 32) z += exp(static_cast<double>(to_f(row[e])) - m);
        z = warp_sum(z);
    }
    for (int k = lane; k < n; k += 32) {
        const int e = held.expert[k];
        const double l = static_cast<double>(to_f(row[e]));
        double v = c.scoring == EXPERTS_SOFTMAX ? exp(l - m) / z : sigmoid(l);
        if (c.bias != nullptr) v += static_cast<double>(c.bias[e]);
        held.rank[k] = rank_of(v);
    }
    __syncwarp();
}
// The J best of those, one after the other: this lane's picks (pick j at lane
// j % 32, in mine[j / 32]).
__device__ __noinline__ void pick_in_64(const Choose &c, const Held &held, int n, int lane, int (&mine)[2]) {
    mine[0] = mine[1] = -1;
    for (int j = 0; j < c.J; ++j) {
        unsigned long long best = 0;
        int at = -1;
        for (int k = lane; k < n; k += 32)
            if (held.rank[k] > best) {  // the first of equal ones: they are in order
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
// The sum in 64 bits of group g's best, of those of `held`.
__device__ __noinline__ double group_in_64(const Choose &c, const Held &held, int n, unsigned g, int lane) {
    unsigned long long first = 0, second = 0, any;
    for (int k = lane; k < n; k += 32)
        if (group_of(c, held.expert[k]) == g) keep_two(held.rank[k], first, second);
    return best_two<unsigned long long, double>(first, second, c.top > 1, &any);
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
    const bool softmax = c.scoring == EXPERTS_SOFTMAX;
    const int e0 = lane * NV;
    float l[NV];
    load_row<T, NV>(row, lane, c.E, c.wide, -INFINITY, l);
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) m = max_or_nan(m, l[i]);
    m = warp_max_f(m);
    const bool wrong = m != m || (softmax && m == INFINITY);
    const bool summed = c.groups > 1 && c.top > 1;  // groups by sums of scores
    float z = 1.0f;
    if (softmax && (c.bias != nullptr || !c.renormalize || summed) && m > -INFINITY) {
        z = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) z += expf(l[i] - m);
        z = warp_sum(z);
    }
    // How far the difference of two scores may be off, in units of 2^-24.  Sigmoid: the exponential is
    // within 4 of its value and the rounding of its argument moves it by 1.44 |l|, of which a quarter and
    // 0.33 at most reach the score; the sum adds 1, the reciprocal 2: 5 a score.  Softmax, of the largest
    // score 1 / z: 4 of its own exponential (expf), less than 1 of the rounding of l - m (x exp(-x) < 0.4),
    // and those of z: 36 of up to 31 sums in a lane and 5 across, 11 of the exponentials (4, and the
    // rounding of l - m at a mean of up to log 1024); 3 of reciprocal and product.
    const float most = softmax ? lt::fast_reciprocal(z) : 1.0f;
    const float slack = softmax ? most * 0x1p-17f : 0x1p-20f;
    float size = 1.0f;  // of what groups' sums add up
    uint32_t key[NV];
    float bias[NV];
    if (c.bias != nullptr) load_row<float, NV>(c.bias, lane, c.E, c.wide_bias, -INFINITY, bias);
    auto score_of = [&](float x) { return softmax ? expf(x - m) * most : sigmoid_about(x); };
    auto value_of = [&](float x, float b) { return __fadd_rn(score_of(x), b); };  // the same bits wherever it is worked out
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        key[i] = 0;
        if (l[i] > -INFINITY && !wrong) {
            const float v = c.bias != nullptr ? value_of(l[i], bias[i]) : l[i];
            if (v > -INFINITY) {
                key[i] = rank_of(v);
                if (c.bias != nullptr) size = fmaxf(size, fabsf(v));
            }
        }
    }
    Held held;
    held.rank = room + static_cast<size_t>(warp) * c.E;
    held.expert = reinterpret_cast<unsigned short *>(room + static_cast<size_t>(CHOOSE_WARPS) * c.E) + warp * c.E;
    if (c.groups > 1) {
        uint32_t total = 0, least = 0;  // lane g: the rank of group g's sum, and of the least value in it
        auto rank = [&](int i) { return summed && c.bias == nullptr && key[i] != 0 ? rank_of(score_of(l[i])) : key[i]; };
        if (c.lanes > 0) {  // a group is `lanes` lanes, a power of two
            uint32_t first = 0, second = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) keep_two(rank(i), first, second);
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
                    if (group_of(c, e0 + i) == static_cast<unsigned>(g)) keep_two(rank(i), first, second);
                const float sum = best_two<uint32_t, float>(first, second, c.top > 1, &any);
                const uint32_t low = c.top > 1 && __popc(__ballot_sync(ALL, first != 0)) + __popc(__ballot_sync(ALL, second != 0)) < 2
                                         ? 0
                                         : rank_of(c.top > 1 ? sum - of_rank(any) : sum);
                if (lane == g && any != 0) {
                    total = rank_of(sum);
                    least = low;
                }
            }
        }
        unsigned keep = kept_groups(c, total, lane);
        const bool stay = (keep >> lane & 1) != 0;
        if (summed || c.bias != nullptr) {
            // in doubt: the groups whose sums are within `width` of the border's other side
            if (c.bias != nullptr) size = warp_max_f(size);
            const float width = 2.0f * slack + 0x1p-21f * size;  // 4 scores; 4 sums with biases, 2 of two values
            const uint32_t low = __reduce_min_sync(ALL, stay ? total : 0xffffffffu);
            const uint32_t out = warp_max(lane < c.groups && !stay ? total : 0u);
            if (out != 0 && !(of_rank(low) - of_rank(out) >= width)) {
                const float v = of_rank(total);
                const unsigned near = __ballot_sync(ALL, lane < c.groups && total != 0 && (stay ? !(v - of_rank(out) >= width) : !(of_rank(low) - v >= width)));
                const int n = bring_together<NV>(held.expert, c.E, e0, lane, [&](int i) {
                    const unsigned g = group_of(c, e0 + i) & 31;
                    // the group's best, and what may be among them: 2 scores, 2 sums with the bias, and what `least` lost
                    const uint32_t bound = __shfl_sync(ALL, least, g);
                    return key[i] != 0 && (near >> g & 1) != 0 && (bound == 0 || !(of_rank(rank(i)) < of_rank(bound) - width));
                });
                values_in_64(c, row, held, n, lane);
                unsigned long long exact = 0;  // lane g
                for (unsigned left = near; left != 0; left &= left - 1) {
                    const int g = __ffs(left) - 1;
                    const double sum = group_in_64(c, held, n, g, lane);
                    if (lane == g) exact = rank_of(sum);
                }
                const int places = __popc(keep & near);
                int before = 0;
                for (unsigned left = near; left != 0; left &= left - 1) {
                    const int g = __ffs(left) - 1;
                    const unsigned long long o = __shfl_sync(ALL, exact, g);
                    before += o > exact || (o == exact && g < lane) ? 1 : 0;
                }
                keep = (keep & ~near) | __ballot_sync(ALL, (near >> lane & 1) != 0 && before < places);
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
    int n = 33;
    if (c.J < 32) {
        // of as many lanes' best as there are picks and one more, the least: a bound
        uint32_t left = best, bound = 0;
        for (int got = 0; got <= c.J;) {
            bound = warp_max(left);
            if (bound == 0) break;
            const unsigned there = __ballot_sync(ALL, left == bound);
            if (left == bound) left = 0;
            got += __popc(there);
        }
        n = bring_together<NV>(pick, 32, e0, lane, [&](int i) { return key[i] != 0 && key[i] >= bound; });
    }
    if (n <= 32) {
        int e = lane < n ? pick[lane] : -1;
        // its value again, as its lane has it
        float le = e >= 0 ? to_f(row[e]) : 0.0f, be = e >= 0 && c.bias != nullptr ? c.bias[e] : 0.0f;
        float v = c.bias != nullptr ? value_of(le, be) : le;
        const uint32_t k = e >= 0 ? rank_of(v) : 0;
        int place = 0;
#pragma unroll 4
        for (int o = 0; o < n; ++o) {
            const uint32_t other = __shfl_sync(ALL, k, o);
            place += other > k || (other == k && o < lane) ? 1 : 0;
        }
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
                doubt = __any_sync(ALL, close && !(le == ln && be == bn));
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
                if (j > 0 && !(last - v >= slack + 0x1p-22f * fabsf(last)))
                    doubt = doubt || !(to_f(row[who]) == to_f(row[last_who]) && c.bias[who] == c.bias[last_who]);
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
    if (doubt) {  // those that may be among the J best, in 64 bits
        const float low = floor - slack - 0x1p-22f * fabsf(floor);
        const int some = bring_together<NV>(held.expert, c.E, e0, lane, [&](int i) { return key[i] != 0 && !(of_rank(key[i]) < low); });
        values_in_64(c, row, held, some, lane);
        pick_in_64(c, held, some, lane, mine);
    }

    // weights of the picks
    float lj[2], w[2];
    float high = -INFINITY;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        lj[s] = mine[s] >= 0 ? to_f(row[mine[s]]) : -INFINITY;
        high = fmaxf(high, lj[s]);
    }
    float sum = 0.0f;
    const int slots = c.J > 32 ? 2 : 1;
    if (c.renormalize) {
        // relative to the largest pick, so that no pick's score is lost below the smallest number
        high = warp_max_f(high);
        const float ref = softmax ? high : fminf(high, 0.0f);
        #pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (s >= slots) break;
            w[s] = softmax || lj[s] < 0.0f ? expf(lj[s] - ref) : 1.0f;
            if (!softmax) w[s] *= lt::fast_reciprocal(1.0f + expf(-fabsf(lj[s])));
            if (mine[s] < 0) w[s] = 0.0f;
            sum += w[s];
        }
        sum = warp_sum(sum);
    }
    const float share = lt::fast_reciprocal(sum);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if (s >= slots) break;
        if (c.renormalize)
            w[s] *= share;
        else
            w[s] = softmax ? expf(lj[s] - m) * most : sigmoid(lj[s]);
        w[s] = wrong ? __int_as_float(0x7fffffff) : mine[s] < 0 ? 0.0f : w[s] * c.scale;
        const int j = s * 32 + lane;
        if (j < c.J) {
            c.chosen[static_cast<long long>(t) * c.J + j] = mine[s];
            c.weights[static_cast<long long>(t) * c.J + j] = w[s];
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
