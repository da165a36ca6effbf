// linear_few.cu -- y = act(x.w + bias) + residual for up to 16 tokens.
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
// FP32: fused multiply-adds, one per token and weight (splitting a weight into
// pieces for the tensor cores costs more than 16 of them: 45 us measured for
// 4096 x 4096 whatever the tokens).
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
template <int N, bool VEC>
__device__ __forceinline__ Words<N / 2> fetch16(const void *p, int left) {
    Words<N / 2> r;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) r.v[i] = 0u;
    if constexpr (VEC) {
        if (left > 0) r = *static_cast<const Words<N / 2> *>(p);
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

// A block has 16 (order 1) or 32 features.
template <typename T, int ORDER, bool VEC>
__global__ void __launch_bounds__(ORDER ? 256 : 512, ORDER ? 2 : 1) few16_kernel(const Few p) {
    constexpr int WARPS = ORDER ? 8 : 16;
    constexpr int TILES = ORDER ? 2 : 4;
    constexpr int STEP = ORDER ? 32 : 16;       // K of a warp's step
    constexpr int UNROLL = VEC ? 4 : 1;  // steps whose loads are in flight together
    constexpr int XN = STEP / 4;                // consecutive K of a thread
    __shared__ float sums[WARPS][16][8 * TILES + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int f0 = blockIdx.x * 8 * TILES;
    const T *x = static_cast<const T *>(p.x), *w = static_cast<const T *>(p.w);
    const int steps = (p.K + STEP - 1) / STEP;
    const int s0 = static_cast<int>(static_cast<long long>(steps) * warp / WARPS);
    const int s1 = static_cast<int>(static_cast<long long>(steps) * (warp + 1) / WARPS);
    const T *x_lo = x + (g < p.T ? g : 0) * p.ldx, *x_hi = x + (g + 8 < p.T ? g + 8 : 0) * p.ldx;
    const int lo_k = g < p.T ? p.K : 0, hi_k = g + 8 < p.T ? p.K : 0;  // a missing token is zeros
    float acc[TILES][4];
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][k] = 0.0f;
    tc::grid_wait();
    for (int s = s0; s < s1; s += UNROLL) {
        Words<ORDER ? 4 : 2> wv[UNROLL][ORDER ? TILES : 4];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int k = (s + u) * STEP + t * XN;
            const bool in = s + u < s1;
            if constexpr (ORDER) {
#pragma unroll
                for (int i = 0; i < TILES; ++i) {
                    const int f = f0 + 8 * i + g;
                    if constexpr (VEC)
                        wv[u][i] = stream<4>(w + f * p.ldw + k, in && f < p.F && k < p.K);
                    else
                        wv[u][i] = fetch16<8, false>(w + f * p.ldw + k, in && f < p.F ? p.K - k : 0);
                }
            } else {
                const int f = f0 + 4 * g;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (VEC)
                        wv[u][i] = stream<2>(w + (k + i) * p.ldw + f, in && k + i < p.K && f < p.F);
                    else
                        wv[u][i] = fetch16<4, false>(w + (k + i) * p.ldw + f, in && k + i < p.K ? p.F - f : 0);
                }
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
    const int token = threadIdx.x / (8 * TILES), col = threadIdx.x % (8 * TILES), f = f0 + col;
    if (token >= p.T || f >= p.F) return;
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) v += sums[i][token][col];
    finish<T>(p, token, f, v);
}

// TT tokens (at least p.T).  Order 1: 8 warps share out K, each lane 4 K of the
// block's 8 features at a time (4 of them for more than 4 tokens).  Order 0: 16 warps; lane (r, q) takes K r of
// four and features 4 q .. 4 q + 3 of the block's 32.
__host__ __device__ constexpr int own32(int tokens) { return tokens > 4 ? 4 : 8; }
template <int ORDER, int TT, bool VEC>
__global__ void __launch_bounds__(ORDER ? 256 : 512, ORDER ? 2 : 1) few32_kernel(const Few p) {
    constexpr int WARPS = ORDER ? 8 : 16;
    constexpr int OWN = ORDER ? own32(TT) : 4;  // features of a thread
    constexpr int FEATURES = ORDER ? OWN : 32;
    constexpr int STEP = ORDER ? 128 : 4;
    constexpr int UNROLL = ORDER ? 1 : TT > 8 ? 2 : !VEC ? 2 : TT > 4 ? 4 : 8;
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

template <typename K>
cudaError_t launch(K kernel, int features, int threads, const Few &p, cudaStream_t stream) {
    return tc::launch(kernel, static_cast<unsigned>((p.F + features - 1) / features), dim3(static_cast<unsigned>(threads)), 0,
                      stream, p);
}
bool aligned(const void *q, long long ld, int element, int bytes) {
    return reinterpret_cast<uintptr_t>(q) % bytes == 0 && ld * element % bytes == 0;
}
template <typename T>
cudaError_t run16(const Few &p, cudaStream_t stream) {
    if (p.order) {
        const bool vec = p.K % 8 == 0 && aligned(p.x, p.ldx, 2, 16) && aligned(p.w, p.ldw, 2, 16);
        return launch(vec ? few16_kernel<T, 1, true> : few16_kernel<T, 1, false>, 16, 256, p, stream);
    }
    const bool vec = p.K % 4 == 0 && p.F % 4 == 0 && aligned(p.x, p.ldx, 2, 8) && aligned(p.w, p.ldw, 2, 8);
    return launch(vec ? few16_kernel<T, 0, true> : few16_kernel<T, 0, false>, 32, 512, p, stream);
}
template <int TT>
cudaError_t run32(const Few &p, cudaStream_t stream) {
    if (p.order) {
        const bool vec = p.K % 4 == 0 && aligned(p.x, p.ldx, 4, 16) && aligned(p.w, p.ldw, 4, 16);
        return launch(vec ? few32_kernel<1, TT, true> : few32_kernel<1, TT, false>, own32(TT), 256, p, stream);
    }
    const bool vec = p.F % 4 == 0 && aligned(p.w, p.ldw, 4, 16);
    return launch(vec ? few32_kernel<0, TT, true> : few32_kernel<0, TT, false>, 32, 512, p, stream);
}

}  // namespace

cudaError_t run(int type, const Few &p, cudaStream_t stream) {
    sg_nvtx::Range r("linear: few tokens");
    if (type == LINEAR_BF16) return run16<__nv_bfloat16>(p, stream);
    if (type == LINEAR_F16) return run16<__half>(p, stream);
    return p.T <= 1 ? run32<1>(p, stream) : p.T <= 4 ? run32<4>(p, stream) : p.T <= 8 ? run32<8>(p, stream) : run32<16>(p, stream);
}

}  // namespace linear_few
