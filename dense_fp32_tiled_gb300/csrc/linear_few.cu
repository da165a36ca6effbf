// linear_few.cu -- y = act(x.w + bias) + residual for up to 16 tokens, and up to 64
// in FP32 or with few weights.
//
// Such a product reads each weight once and does next to nothing with it, so
// what counts is that loads of the weight start at once and keep coming: no
// tensor copies, barriers, tensor memory or clusters to set up, but wide loads
// straight into registers, eight or more in flight per thread, with the K
// shared out over a block's warps, whose sums meet in shared memory and are
// added in warp order.
//
// 16-bit types: mma.sync fragments of 16 tokens x 8 features x 16 K.  The K of a
// fragment may be any 16 as long as both operands agree on them, so a thread's
// consecutive values serve as its fragment's as they come:
//   order 1 (K contiguous): thread (g, t) of a warp takes the 8 K from 8 t on
//     of feature g, which are its share of two fragments (32 K).
//   order 0 (features contiguous): it takes features 4 g .. 4 g + 3 of the four
//     K from 4 t on, paired up in registers into the shares of four fragments
//     (features 4 g + i for fragment i).
// FP32, up to 4 tokens: fused multiply-adds, one per token and weight (4 x 8192 x
// 8192 50 us; on the tensor cores 54).  More tokens: mma.sync on three bf16 pieces
// that each warp makes of its values in registers, so that the weight is read once
// in FP32, where the product kernel's operand copies read 4 bytes of it and write
// and read 6.  us, K contiguous, multiply-adds / product kernel / this:
//   8 x 4096^2 24 / 54 / 18.1      16 x 4096^2 38 / 54 / 22.8  16 x 8192^2 107 / 180 / 66.7
//   32 x 4096^2 - / 55 / 27.5      32 x 8192^2 - / 183 / 92.3  48 x 8192^2 - / 186 / 128
//   64 x 4096^2 - / 57 / 52.7      64 x 8192^2 - / 186 / 185   64 x 1000 x 1024 - / 19 / 10.5
// mma.sync bounds it from about 16 tokens on (10 to 12 cycles a scheduler for each).
#include "linear_few.cuh"

#include <cstdint>
#include <type_traits>

#include "linear_types.cuh"
#include "nvtx_range.cuh"
#include "tensor_core.cuh"

namespace linear_few {
namespace {

using lt::from_f;
using lt::to_f;

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
            "%2, %3};\n"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, "
            "%1, %2, %3};\n"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// N consecutive values, `left` of them in the matrix (the others 0).  VEC: one
// aligned load, all or nothing (sizes are multiples of N), so that it is a
// predicated instruction and nothing keeps the next ones from following at once.
// fetch16 has a form for even sizes between: 2, by pairs of values.
template <int WORDS>
struct alignas(4 * WORDS) Words {
    uint32_t v[WORDS];
};
// A weight's 16 or 8 bytes, read once: not kept in L1, and L2 fetches the 256
// bytes around them at once, which other steps of the warp (order 0: the
// neighbouring blocks) read next, as an access takes only 64 bytes of a row (one
// token, 8192 x 8192, 16 bits: 30 us without, 25 with).  Volatile keeps it behind
// grid_wait.
template <int WORDS>
__device__ __forceinline__ Words<WORDS> stream(const void *p, bool in) {
    Words<WORDS> r;
#pragma unroll
    for (int i = 0; i < WORDS; ++i) r.v[i] = 0u;
    if (in) {
        if constexpr (WORDS == 4)
            asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                         : "=r"(r.v[0]), "=r"(r.v[1]), "=r"(r.v[2]), "=r"(r.v[3])
                         : "l"(p));
        else
            asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v2.b32 {%0, %1}, [%2];\n" : "=r"(r.v[0]), "=r"(r.v[1]) : "l"(p));
    }
    return r;
}
template <int N, int VEC>
__device__ __forceinline__ Words<N / 2> fetch16(const void *p, int left) {
    Words<N / 2> r;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) r.v[i] = 0u;
    if constexpr (VEC == 1) {
        if (left > 0) r = *static_cast<const Words<N / 2> *>(p);
    } else if constexpr (VEC == 2) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            if (2 * i < left) r.v[i] = static_cast<const uint32_t *>(p)[i];
    } else {
        const unsigned short *q = static_cast<const unsigned short *>(p);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < left) r.v[i / 2] |= static_cast<uint32_t>(q[i]) << (16 * (i & 1));
    }
    return r;
}
template <bool VEC>
__device__ __forceinline__ float4 fetch32(const float *p, int left) {
    float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if constexpr (VEC) {
        if (left > 0) r = *reinterpret_cast<const float4 *>(p);
    } else {
        if (left > 0) r.x = p[0];
        if (left > 1) r.y = p[1];
        if (left > 2) r.z = p[2];
        if (left > 3) r.w = p[3];
    }
    return r;
}

// fetch32 for a weight, see stream
template <bool VEC>
__device__ __forceinline__ float4 stream32(const float *p, int left) {
    if constexpr (!VEC) return fetch32<false>(p, left);
    const Words<4> r = stream<4>(p, left > 0);
    return make_float4(__uint_as_float(r.v[0]), __uint_as_float(r.v[1]), __uint_as_float(r.v[2]), __uint_as_float(r.v[3]));
}

template <typename T>
__device__ __forceinline__ void finish(const Few &p, int token, int f, float v) {
    if (p.bias != nullptr) v += to_f(static_cast<const T *>(p.bias)[f]);
    if (p.z != nullptr) static_cast<T *>(p.z)[token * p.ldz + f] = from_f<T>(v);
    lt::with_activation(p.act, [&](auto a) { v = lt::activate<decltype(a)::value, std::is_same<T, float>::value>(v); });
    if (p.residual != nullptr) v += to_f(static_cast<const T *>(p.residual)[token * p.ldr + f]);
    static_cast<T *>(p.out)[token * p.ldo + f] = from_f<T>(v);
}

// A cluster's CTAs add their sums of a tile in order of their rank, each for its
// share of the outputs.
template <typename T, int THREADS, int TOKENS, int FEATURES>
__device__ __forceinline__ void join(const Few &p, const float (&own)[TOKENS][FEATURES], int f0, int rank) {
    tc::cluster_sync();
    for (int o = rank * THREADS + threadIdx.x; o < TOKENS * FEATURES; o += p.split * THREADS) {
        const int token = o / FEATURES, col = o % FEATURES, f = f0 + col;
        if (token >= p.T || f >= p.F) continue;
        float v = 0.0f;
        for (int r = 0; r < p.split; ++r) v += tc::ld_cluster_f32(tc::peer_addr(tc::smem_u32(&own[token][col]), r));
        finish<T>(p, token, f, v);
    }
    tc::cluster_sync();  // no CTA ends while another reads its sums
}

// A block has 16 (order 1) or 32 features.
template <typename T, int ORDER, int WARPS, int VEC, bool SPLIT>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) few16_kernel(const Few p) {
    constexpr int TILES = ORDER ? 2 : 4;
    constexpr int STEP = ORDER ? 32 : 16;                        // K of a warp's step
    constexpr int UNROLL = VEC == 1 ? 4 : 1;              // steps whose loads are in flight together
    constexpr int ROWS = ORDER ? TILES : 4;                      // loads of a thread's step
    constexpr int XN = STEP / 4;                                 // consecutive K of a thread
    constexpr int FEATURES = 8 * TILES;
    __shared__ float sums[WARPS][16][FEATURES + 1];
    __shared__ float own[16][FEATURES];  // this CTA's sums, for its cluster
    const int split = SPLIT ? p.split : 1, rank = blockIdx.x % split;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int f0 = static_cast<int>(blockIdx.x / split) * FEATURES;
    const T *x = static_cast<const T *>(p.x), *w = static_cast<const T *>(p.w);
    const int steps = (p.K + STEP - 1) / STEP;
    const int s0 = static_cast<int>(static_cast<long long>(steps) * (rank * WARPS + warp) / (WARPS * split));
    const int s1 = static_cast<int>(static_cast<long long>(steps) * (rank * WARPS + warp + 1) / (WARPS * split));
    const T *x_lo = x + (g < p.T ? g : 0) * p.ldx, *x_hi = x + (g + 8 < p.T ? g + 8 : 0) * p.ldx;
    const int lo_k = g < p.T ? p.K : 0, hi_k = g + 8 < p.T ? p.K : 0;  // a missing token is zeros
    float acc[TILES][4];
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][k] = 0.0f;
    tc::grid_wait();
    for (int s = s0; s < s1; s += UNROLL) {
        Words<ORDER ? 4 : 2> wv[UNROLL][ROWS];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int k = (s + u) * STEP + t * XN;
            const bool in = s + u < s1;
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const int f = ORDER ? f0 + 8 * i + g : f0 + 4 * g, kk = ORDER ? k : k + i;
                const T *q = w + (ORDER ? f * p.ldw + kk : kk * p.ldw + f);
                const bool here = in && f < p.F && kk < p.K;
                if constexpr (VEC == 1)
                    wv[u][i] = stream<ORDER ? 4 : 2>(q, here);
                else
                    wv[u][i] = fetch16<ORDER ? 8 : 4, VEC>(q, here ? ORDER ? p.K - kk : p.F - f : 0);
            }
        }
        Words<XN / 2> lo[UNROLL], hi[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int k = (s + u) * STEP + t * XN;
            const bool in = s + u < s1;
            lo[u] = fetch16<XN, VEC>(x_lo + k, in ? lo_k - k : 0);
            hi[u] = fetch16<XN, VEC>(x_hi + k, in ? hi_k - k : 0);
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
#pragma unroll
            for (int h = 0; h < STEP / 16; ++h) {  // fragments of 16 K
                const uint32_t a[4] = {lo[u].v[2 * h], hi[u].v[2 * h], lo[u].v[2 * h + 1], hi[u].v[2 * h + 1]};
#pragma unroll
                for (int i = 0; i < TILES; ++i) {
                    if constexpr (ORDER) {
                        mma<T>(acc[i], a, wv[u][i].v[2 * h], wv[u][i].v[2 * h + 1]);
                    } else {  // value i of rows 0, 1 and of rows 2, 3
                        const uint32_t sel = i & 1 ? 0x7632 : 0x5410;
                        mma<T>(acc[i], a, __byte_perm(wv[u][0].v[i / 2], wv[u][1].v[i / 2], sel),
                               __byte_perm(wv[u][2].v[i / 2], wv[u][3].v[i / 2], sel));
                    }
                }
            }
    }
    // fragment (g, t): tokens g and g + 8, columns 2 t and 2 t + 1 of each tile
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int n = 2 * t + (k & 1);
            sums[warp][g + 8 * (k >> 1)][ORDER ? 8 * i + n : 4 * n + i] = acc[i][k];
        }
    __syncthreads();
#pragma unroll
    for (int o = threadIdx.x; o < 16 * FEATURES; o += WARPS * 32) {
        const int token = o / FEATURES, col = o % FEATURES, f = f0 + col;
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) v += sums[i][token][col];
        if (SPLIT)
            own[token][col] = v;
        else if (token < p.T && f < p.F)
            finish<T>(p, token, f, v);
    }
    if (SPLIT) join<T, WARPS * 32>(p, own, f0, rank);
}

// TT tokens (at least p.T).  Order 1: 8 warps share out K, each lane 4 K of the
// block's 8 features at a time.  Order 0: 16 warps; lane (r, q) takes K r of four
// and features 4 q .. 4 q + 3 of the block's 32.
template <int ORDER, int TT, bool VEC>
__global__ void __launch_bounds__(ORDER ? 256 : 512, ORDER ? 2 : 1) few32_kernel(const Few p) {
    constexpr int WARPS = ORDER ? 8 : 16;
    constexpr int OWN = ORDER ? 8 : 4;  // features of a thread
    constexpr int FEATURES = ORDER ? OWN : 32;
    constexpr int STEP = ORDER ? 128 : 4;
    constexpr int UNROLL = ORDER ? 1 : VEC ? 8 : 2;
    __shared__ float sums[WARPS][TT][FEATURES];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int f0 = blockIdx.x * FEATURES;
    const float *x = static_cast<const float *>(p.x), *w = static_cast<const float *>(p.w);
    const int steps = (p.K + STEP - 1) / STEP;
    const int s0 = static_cast<int>(static_cast<long long>(steps) * warp / WARPS);
    const int s1 = static_cast<int>(static_cast<long long>(steps) * (warp + 1) / WARPS);
    float acc[TT][OWN];
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int k = 0; k < OWN; ++k) acc[i][k] = 0.0f;
    tc::grid_wait();
    for (int s = s0; s < s1; s += UNROLL) {
        if constexpr (ORDER) {
            const int k = s * STEP + 4 * lane;
            float4 wv[OWN];
#pragma unroll
            for (int i = 0; i < OWN; ++i) wv[i] = stream32<VEC>(w + (f0 + i) * p.ldw + k, f0 + i < p.F ? p.K - k : 0);
#pragma unroll
            for (int j = 0; j < TT; ++j) {
                const float4 xv = fetch32<VEC>(x + j * p.ldx + k, j < p.T ? p.K - k : 0);
#pragma unroll
                for (int i = 0; i < OWN; ++i)
                    acc[j][i] = fmaf(xv.w, wv[i].w, fmaf(xv.z, wv[i].z, fmaf(xv.y, wv[i].y, fmaf(xv.x, wv[i].x, acc[j][i]))));
            }
        } else {
            const int r = lane >> 3, f = f0 + 4 * (lane & 7);
            float4 wv[UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int k = (s + u) * STEP + r;
                wv[u] = stream32<VEC>(w + k * p.ldw + f, s + u < s1 && k < p.K ? p.F - f : 0);
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int k = (s + u) * STEP + r;
#pragma unroll
                for (int j = 0; j < TT; ++j) {
                    const float xv = j < p.T && s + u < s1 && k < p.K ? x[j * p.ldx + k] : 0.0f;
                    acc[j][0] = fmaf(xv, wv[u].x, acc[j][0]);
                    acc[j][1] = fmaf(xv, wv[u].y, acc[j][1]);
                    acc[j][2] = fmaf(xv, wv[u].z, acc[j][2]);
                    acc[j][3] = fmaf(xv, wv[u].w, acc[j][3]);
                }
            }
        }
    }
    // a warp's sum over its lanes (order 0: those of the same features)
#pragma unroll
    for (int j = 0; j < TT; ++j)
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            float v = acc[j][i];
#pragma unroll
            for (int d = 16; d >= (ORDER ? 1 : 8); d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
            if (ORDER ? lane == 0 : lane < 8) sums[warp][j][ORDER ? i : 4 * lane + i] = v;
        }
    __syncthreads();
    for (int o = threadIdx.x; o < TT * FEATURES; o += WARPS * 32) {
        const int token = o / FEATURES, col = o % FEATURES, f = f0 + col;
        if (token >= p.T || f >= p.F) continue;
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) v += sums[i][token][col];
        finish<float>(p, token, f, v);
    }
}

// The warps' sums of 32 features as rows (rows 2 i and 2 i + 1 of a thread are
// fragment i's rows g and g + 8: features g + 8 r, order 0: 4 g + r), 8 NT tokens
// as columns, added in order of the warps, two tiles of tokens at a time.
template <typename T, int ORDER, int NT, int WARPS, bool SPLIT>
__device__ __forceinline__ void add_warps(const Few &p, const float (&total)[NT][2][4], int f0, int rank) {
    constexpr int PAIR = NT > 1 ? 2 : 1;
    __shared__ float sums[WARPS][8 * PAIR][33];
    __shared__ float own[8 * NT][32];  // this CTA's sums, for its cluster
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int j = 0; j < NT; j += PAIR) {
        if (j > 0) __syncthreads();
#pragma unroll
        for (int q = 0; q < PAIR; ++q)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = 2 * i + (k >> 1);
                    sums[warp][8 * q + 2 * t + (k & 1)][ORDER ? g + 8 * r : 4 * g + r] = total[j + q][i][k];
                }
        __syncthreads();
        for (int o = threadIdx.x; o < 8 * PAIR * 32; o += WARPS * 32) {
            const int token = 8 * j + o / 32, col = o % 32, f = f0 + col;
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < WARPS; ++i) v += sums[i][o / 32][col];
            if (SPLIT)
                own[token][col] = v;
            else if (token < p.T && f < p.F)
                finish<T>(p, token, f, v);
        }
    }
    if (SPLIT) join<T, WARPS * 32>(p, own, f0, rank);
}

// 16-bit types, 17 to 64 tokens (see takes): features as rows, so that a fragment of the weight
// serves all tokens, 8 NT of them as columns.  A warp's step is 32 features x 32 K;
// a thread's K are the eight from 8 t on, four for each of two fragments' columns:
//   order 1: features g + 8 r, r = 0 .. 3, each by 16 bytes of K
//   order 0: features 4 g + r, by 8 bytes of features for each K, paired up
template <typename T, int ORDER, int NT, bool SPLIT>
__global__ void __launch_bounds__(256, NT <= 4 ? 2 : 1) rows16_kernel(const Few p) {
    constexpr int WARPS = 8, DEPTH = 2;
    const int split = SPLIT ? p.split : 1, rank = blockIdx.x % split;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int f0 = static_cast<int>(blockIdx.x / split) * 32;
    const T *x = static_cast<const T *>(p.x) + g * p.ldx + 8 * t, *w = static_cast<const T *>(p.w);
    const int steps = (p.K + 31) / 32;
    const int s0 = static_cast<int>(static_cast<long long>(steps) * (rank * WARPS + warp) / (WARPS * split));
    const int s1 = static_cast<int>(static_cast<long long>(steps) * (rank * WARPS + warp + 1) / (WARPS * split));
    w += ORDER ? (f0 + g) * p.ldw + 8 * t : f0 + 4 * g + 8 * t * p.ldw;
    uint32_t wv[DEPTH][16];
    Words<4> xv[DEPTH][NT];
    float acc[NT][2][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j][i >> 2][i & 3] = 0.0f;
    auto load = [&](int s, int d) {
        const bool in = s < s1 && 32 * s + 8 * t < p.K;
        if constexpr (ORDER) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const Words<4> v = stream<4>(w + 8 * r * p.ldw + 32 * s, in && f0 + g + 8 * r < p.F);
#pragma unroll
                for (int q = 0; q < 4; ++q) wv[d][4 * r + q] = v.v[q];
            }
        } else {
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const Words<2> v = stream<2>(w + (32ll * s + r) * p.ldw, in && f0 + 4 * g < p.F);
                wv[d][2 * r] = v.v[0], wv[d][2 * r + 1] = v.v[1];
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) xv[d][j] = fetch16<8, 1>(x + 8 * j * p.ldx + 32 * s, in && 8 * j + g < p.T ? 8 : 0);
    };
    // K 8 t + 4 h + 2 pair and the next one of row r
    auto value = [&](int d, int h, int r, int pair) {
        if constexpr (ORDER) {
            return wv[d][4 * r + 2 * h + pair];
        } else {
            const int k = 4 * h + 2 * pair;
            return __byte_perm(wv[d][2 * k + r / 2], wv[d][2 * k + 2 + r / 2], r & 1 ? 0x7632 : 0x5410);
        }
    };
    tc::grid_wait();
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(s0 + d, d);
    for (int s = s0; s < s1; s += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t a[4] = {value(d, h, 2 * i, 0), value(d, h, 2 * i + 1, 0), value(d, h, 2 * i, 1),
                                           value(d, h, 2 * i + 1, 1)};
#pragma unroll
                    for (int j = 0; j < NT; ++j) mma<T>(acc[j][i], a, xv[d][j].v[2 * h], xv[d][j].v[2 * h + 1]);
                }
            load(s + DEPTH + d, d);
        }
    }
    add_warps<T, ORDER, NT, WARPS, SPLIT>(p, acc, f0, rank);
}

// FP32, more than four tokens: mma.sync on the three bf16 pieces that the warp
// makes of its values, six products, features as rows and tokens as
// columns (8 NT of them).  A warp's step is 32 features x 16 K; the K of a
// fragment are a thread's four from 4 t on, and its rows:
//   order 1: features g + 8 r, r = 0 .. 3, each by its own 16 bytes of K
//   order 0: features 4 g + r, by 16 bytes of features for each K
// rows 2 i and 2 i + 1 being fragment i's rows g and g + 8.  128 K are summed on
// the tensor cores, those sums in FP32.
// Where there are few features a cluster of up to 8 CTAs shares a tile's K (SPLIT)
// and adds their sums in order of their rank: 32 x 256 x 8192 49 -> 12.6 us.
template <int NT>
struct FewTile {
    static constexpr int WARPS = NT <= 2 ? 16 : 8;   // accumulators: 16 NT registers
    static constexpr int DEPTH = NT <= 4 ? 2 : 1;    // steps whose loads are in flight
};
// x and y as three bf16 pieces each (x in the low halves), each rounded to nearest,
// two values an instruction: x = a + b + c to 2^-27, and the products left out are
// about 2^-24 of the full one at most, either way.  (Cut by masks, that is 2^-21, always
// towards zero.  us, cut / rounded: K contiguous 16 x 8192^2 59 / 60, 32 x 8192^2 94 / 89,
// 64 x 4096^2 46 / 47; features contiguous 63 / 70, 96 / 103, 48 / 45.)  The first piece
// stops at bf16's largest value where rounding would overflow; an infinity passes into the
// second, and the third is a NaN.
__device__ __forceinline__ void pieces2(float x, float y, uint32_t (&r)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (i == 0)
            asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;\n" : "=r"(r[i]) : "f"(y), "f"(x));
        else
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r[i]) : "f"(y), "f"(x));
        x -= __uint_as_float(r[i] << 16);
        y -= __uint_as_float(r[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ float part(const float4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

template <int ORDER, int NT, bool VEC, bool SPLIT>
__global__ void __launch_bounds__(FewTile<NT>::WARPS * 32, 1) few32_mma_kernel(const Few p) {
    constexpr int WARPS = FewTile<NT>::WARPS, DEPTH = FewTile<NT>::DEPTH;
    const int split = SPLIT ? p.split : 1;
    constexpr int PAIR = NT > 1 ? 2 : 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rank = blockIdx.x % split, f0 = static_cast<int>(blockIdx.x / split) * 32;
    const float *x = static_cast<const float *>(p.x) + g * p.ldx + 4 * t, *w = static_cast<const float *>(p.w);
    const int steps = (p.K + 15) / 16;
    const int s0 = static_cast<int>(static_cast<long long>(steps) * (rank * WARPS + warp) / (WARPS * split));
    const int s1 = static_cast<int>(static_cast<long long>(steps) * (rank * WARPS + warp + 1) / (WARPS * split));
    w += ORDER ? (f0 + g) * p.ldw + 4 * t : f0 + 4 * g + 4 * t * p.ldw;
    float4 wv[DEPTH][4], xv[DEPTH][NT];
    float acc[NT][2][4], total[NT][2][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j][i >> 2][i & 3] = total[j][i >> 2][i & 3] = 0.0f;
    auto load = [&](int s, int d) {
        const int k = 16 * s + 4 * t;
        const bool in = s < s1;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if constexpr (ORDER)
                wv[d][r] = stream32<VEC>(w + 8 * r * p.ldw + 16 * s, in && f0 + g + 8 * r < p.F ? p.K - k : 0);
            else
                wv[d][r] = stream32<VEC>(w + (16ll * s + r) * p.ldw, in && k + r < p.K ? p.F - (f0 + 4 * g) : 0);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) xv[d][j] = fetch32<VEC>(x + 8 * j * p.ldx + 16 * s, in && 8 * j + g < p.T ? p.K - k : 0);
    };
    tc::grid_wait();
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(s0 + d, d);
    for (int s = s0; s < s1; s += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            uint32_t a[2][4][3];  // fragment, register, piece
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    pieces2(ORDER ? part(wv[d][r], 2 * h) : part(wv[d][2 * h], r),
                            ORDER ? part(wv[d][r], 2 * h + 1) : part(wv[d][2 * h + 1], r), a[r >> 1][(r & 1) + 2 * h]);
#pragma unroll
            for (int j = 0; j < NT; j += PAIR) {
                uint32_t b[PAIR][2][3];
#pragma unroll
                for (int q = 0; q < PAIR; ++q) {
                    pieces2(xv[d][j + q].x, xv[d][j + q].y, b[q][0]);
                    pieces2(xv[d][j + q].z, xv[d][j + q].w, b[q][1]);
                }
                constexpr int WP[6] = {2, 0, 1, 1, 0, 0}, XP[6] = {0, 2, 1, 0, 1, 0};  // the small products first
#pragma unroll
                for (int m = 0; m < 6; ++m)
#pragma unroll
                    for (int q = 0; q < PAIR; ++q)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t av[4] = {a[i][0][WP[m]], a[i][1][WP[m]], a[i][2][WP[m]], a[i][3][WP[m]]};
                            mma<__nv_bfloat16>(acc[j + q][i], av, b[q][0][XP[m]], b[q][1][XP[m]]);
                        }
            }
            load(s + DEPTH + d, d);
        }
        if ((s - s0) % 8 == 8 - DEPTH || s + DEPTH >= s1) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    total[j][i >> 2][i & 3] += acc[j][i >> 2][i & 3];
                    acc[j][i >> 2][i & 3] = 0.0f;
                }
        }
    }
    add_warps<float, ORDER, NT, WARPS, SPLIT>(p, total, f0, rank);
}

template <typename K>
cudaError_t launch(K kernel, int features, int threads, const Few &p, cudaStream_t stream) {
    return tc::launch(kernel, static_cast<unsigned>((p.F + features - 1) / features), dim3(static_cast<unsigned>(threads)), 0,
                      stream, p);
}
bool aligned(const void *q, long long ld, int element, int bytes) {
    return reinterpret_cast<uintptr_t>(q) % bytes == 0 && ld * element % bytes == 0;
}
// CTAs that share a tile's K: as many as find room at once, at most a portable
// cluster's 8, each of their warps keeping `least` steps (16 x 2048 x 11008 bf16
// 22 -> 16.7 us, K contiguous 15.6 -> 14.1; 1 x 256 x 8192 15.6 -> 6.7 and 10.8 ->
// 6.7; with half the steps 1 x 2048 x 2048 took 6.6 us for 5.8).
int shares(long long tiles, long long places, long long steps, int warps, int least) {
    int split = 1;
    while (split < 8 && 2 * split * tiles <= places && steps >= 2ll * split * warps * least) split *= 2;
    return split;
}
template <typename T, int ORDER, int WARPS, bool SPLIT>
cudaError_t launch16(int vec, const Few &p, long long tiles, cudaStream_t stream) {
    return tc::launch_clusters(vec == 1   ? few16_kernel<T, ORDER, WARPS, 1, SPLIT>
                               : vec == 2 ? few16_kernel<T, ORDER, WARPS, 2, SPLIT>
                                          : few16_kernel<T, ORDER, WARPS, 0, SPLIT>,
                               SPLIT ? static_cast<unsigned>(p.split) : 1u, static_cast<unsigned>(tiles * p.split),
                               dim3(WARPS * 32), 0, stream, p);
}
// Whether the operands can be read by n values of K of x, and of w's rows.
bool read_by(const Few &p, int n) {
    return p.K % n == 0 && (p.order || p.F % n == 0) && aligned(p.x, p.ldx, 2, 2 * n) && aligned(p.w, p.ldw, 2, 2 * n);
}
template <typename T, int ORDER, int NT>
cudaError_t rows16(Few p, cudaStream_t stream) {
    const long long tiles = (p.F + 31ll) / 32;
    p.split = shares(tiles, p.sms, (p.K + 31ll) / 32, 8, 2);
    return tc::launch_clusters(p.split > 1 ? rows16_kernel<T, ORDER, NT, true> : rows16_kernel<T, ORDER, NT, false>,
                               static_cast<unsigned>(p.split), static_cast<unsigned>(tiles * p.split), dim3(256), 0, stream, p);
}
template <typename T, int ORDER>
cudaError_t rows16(const Few &p, cudaStream_t stream) {
    return p.T <= 32 ? rows16<T, ORDER, 4>(p, stream) : rows16<T, ORDER, 8>(p, stream);
}
template <typename T>
cudaError_t run16(Few p, cudaStream_t stream) {
    if (p.T > 16) return p.order ? rows16<T, 1>(p, stream) : rows16<T, 0>(p, stream);
    const int vec = read_by(p, p.order ? 8 : 4) ? 1 : read_by(p, 2) ? 2 : 0;
    if (p.order) {
        const long long tiles = (p.F + 15ll) / 16;
        p.split = shares(tiles, 2ll * p.sms, (p.K + 31ll) / 32, 8, 8);
        return p.split > 1 ? launch16<T, 1, 8, true>(vec, p, tiles, stream) : launch16<T, 1, 8, false>(vec, p, tiles, stream);
    }
    // 16 warps while each tile has an SM (1 x 4096 x 4096 11.1 us, with 8 warps and
    // twice the shares of K 12.2), else 8, two blocks an SM (1 x 8192 x 8192 29; 34)
    const long long tiles = (p.F + 31ll) / 32;
    p.split = 1;
    if (tiles > p.sms) return launch16<T, 0, 8, false>(vec, p, tiles, stream);
    p.split = shares(tiles, p.sms, (p.K + 15ll) / 16, 16, 4);
    return p.split > 1 ? launch16<T, 0, 16, true>(vec, p, tiles, stream) : launch16<T, 0, 16, false>(vec, p, tiles, stream);
}
template <int TT>
cudaError_t run32(const Few &p, cudaStream_t stream) {
    if (p.order) {
        const bool vec = p.K % 4 == 0 && aligned(p.x, p.ldx, 4, 16) && aligned(p.w, p.ldw, 4, 16);
        return launch(vec ? few32_kernel<1, TT, true> : few32_kernel<1, TT, false>, 8, 256, p, stream);
    }
    const bool vec = p.F % 4 == 0 && aligned(p.w, p.ldw, 4, 16);
    return launch(vec ? few32_kernel<0, TT, true> : few32_kernel<0, TT, false>, 32, 512, p, stream);
}
template <int ORDER, int NT>
cudaError_t run32_mma(bool vec, Few p, cudaStream_t stream) {
    constexpr int WARPS = FewTile<NT>::WARPS;
    const long long tiles = (p.F + 31ll) / 32, steps = (p.K + 15ll) / 16;
    p.split = shares(tiles, p.sms, steps, WARPS, FewTile<NT>::DEPTH);
    const auto kernel = p.split > 1 ? (vec ? few32_mma_kernel<ORDER, NT, true, true> : few32_mma_kernel<ORDER, NT, false, true>)
                                    : (vec ? few32_mma_kernel<ORDER, NT, true, false> : few32_mma_kernel<ORDER, NT, false, false>);
    return tc::launch_clusters(kernel, static_cast<unsigned>(p.split), static_cast<unsigned>(tiles * p.split),
                               dim3(WARPS * 32), 0, stream, p);
}
template <int NT>
cudaError_t run32_mma(const Few &p, cudaStream_t stream) {
    const bool vec = p.K % 4 == 0 && aligned(p.x, p.ldx, 4, 16) && aligned(p.w, p.ldw, 4, 16);
    return p.order ? run32_mma<1, NT>(vec, p, stream) : run32_mma<0, NT>(vec && p.F % 4 == 0, p, stream);
}

}  // namespace

// More than 16 tokens.  FP32: beyond 64, splitting the operands once for the product
// kernel costs less than in each CTA.  16 bits: each CTA reads all of x, so the
// product kernel, about 10 us whatever its size, is left behind only below about
// 8 million weights (us, product kernel / rows16_kernel: 32 x 512 x 512 11.0 / 5.5,
// 24 x 1024 x 1024 11.2 / 7.2, 32 x 256 x 8192 17.9 / 8.2, 48 x 2048 x 2048 12.9 /
// 10.5; 48 x 4096 x 4096 16.4 / 17.0, 64 x 8192 x 8192 32 / 59).
bool takes(int type, const Few &p) {
    if (p.T <= 16) return true;
    if (type == LINEAR_F32) return p.T <= 64;
    return p.T <= 64 && static_cast<long long>(p.F) * p.K <= 1 << 23 && p.K % 8 == 0 && (p.order || p.F % 8 == 0) &&
           aligned(p.x, p.ldx, 2, 16) && aligned(p.w, p.ldw, 2, 16);
}

cudaError_t run(int type, const Few &p, cudaStream_t stream) {
    sg_nvtx::Range r("linear: few tokens");
    if (type == LINEAR_BF16) return run16<__nv_bfloat16>(p, stream);
    if (type == LINEAR_F16) return run16<__half>(p, stream);
    if (p.T <= 4) return p.T <= 1 ? run32<1>(p, stream) : run32<4>(p, stream);
    if (p.T <= 16) return p.T <= 8 ? run32_mma<1>(p, stream) : run32_mma<2>(p, stream);
    return p.T <= 32 ? run32_mma<4>(p, stream) : p.T <= 48 ? run32_mma<6>(p, stream) : run32_mma<8>(p, stream);
}

}  // namespace linear_few
