// linear_prep.cu -- see linear_prep.cuh.
#include "linear_prep.cuh"

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "linear_types.cuh"
#include "nvtx_range.cuh"
#include "tensor_core.cuh"

namespace {

using lt::from_f;
using lt::pieces;
using lt::to_f;

template <typename T>
struct alignas(sizeof(T) * 8) Vec8 {
    T v[8];
};
template <typename T>
struct alignas(16) Chunk {  // 16 bytes
    T v[16 / sizeof(T)];
};

// 8 consecutive values per thread and step.  Bound by HBM: 4 bytes read and 6
// written per FP32 value (4096 x 4096: 25 us, 6.7 TB/s).
struct Job {
    linear_prep::Copy c;
    long long units;  // groups of 8
    int vec;          // aligned 16-byte loads
};
template <typename T>
__device__ __forceinline__ void copy8(const Job &job, long long u) {
    const linear_prep::Copy &m = job.c;
    const int per_row = (m.inner + 7) / 8;
    const long long row = u / per_row;
    const int j = static_cast<int>(u - row * per_row) * 8;
    const long long e = row / m.outer;
    const T *s = static_cast<const T *>(m.src) + e * m.plane + (row - e * m.outer) * m.ld + j;
    T v[8];
    if (job.vec && j + 8 <= m.inner) {
#pragma unroll
        for (int i = 0; i < 8; i += 16 / static_cast<int>(sizeof(T))) {
            const Chunk<T> c = *reinterpret_cast<const Chunk<T> *>(s + i);
#pragma unroll
            for (int k = 0; k < 16 / static_cast<int>(sizeof(T)); ++k) v[i + k] = c.v[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = j + i < m.inner ? s[i] : from_f<T>(0.0f);
    }
    if constexpr (std::is_same<T, float>::value) {
        Vec8<__nv_bfloat16> a, b, c;
#pragma unroll
        for (int i = 0; i < 8; ++i) pieces(v[i], a.v[i], b.v[i], c.v[i]);
        auto *d = static_cast<Vec8<__nv_bfloat16> *>(m.dst);
        d[u] = a;
        d[job.units + u] = b;
        d[2 * job.units + u] = c;
    } else {
        Vec8<T> o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o.v[i] = v[i];
        static_cast<Vec8<T> *>(m.dst)[u] = o;
    }
}
template <typename T>
__global__ void __launch_bounds__(256) copy_operands_kernel(const Job a, const Job b) {
    tc::grid_trigger();  // the next kernel may set itself up meanwhile; it waits for this grid before it reads
    tc::grid_wait();
    const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
    for (long long u = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; u < a.units + b.units; u += step) {
        if (u < a.units)
            copy8<T>(a, u);
        else
            copy8<T>(b, u - a.units);
    }
}

template <typename T>
Job job_of(const linear_prep::Copy &c) {
    const int n = 16 / static_cast<int>(sizeof(T));
    Job j;
    j.c = c;
    j.units = static_cast<long long>(c.planes) * c.outer * ((c.inner + 7) / 8);
    j.vec = reinterpret_cast<uintptr_t>(c.src) % 16 == 0 && c.ld % n == 0 && (c.planes <= 1 || c.plane % n == 0);
    return j;
}
template <typename T>
cudaError_t copy_operands_t(const linear_prep::Copy *copies, int n, cudaStream_t stream) {
    const Job a = job_of<T>(copies[0]);
    Job b = a;
    b.units = 0;
    if (n > 1) b = job_of<T>(copies[1]);
    long long blocks = (a.units + b.units + 255) / 256;
    if (blocks > 152 * 64) blocks = 152 * 64;
    return tc::launch(copy_operands_kernel<T>, static_cast<unsigned>(blocks), dim3(256), 0, stream, a, b);
}

// ---- dz = dy * act'(z), and its column sums -------------------------------------------
// dz of the 16-bit types is rounded to them, as a chain of 16-bit tensors would hold it:
// dx and dw are then 2.35e-3 off in the root mean square in bf16, 2.9e-4 in float16
// (rounded once 1.66e-3 and 2.1e-4).  A second piece of dz would take both products twice.
// A block takes a chunk of rows of 32 * V columns; warp w its rows w, w + 8, ...
// Rows of different experts are summed apart; the chunks' sums are added up
// afterwards, in chunk order, so they do not depend on timing.
using linear_prep::CHUNK;
constexpr int GWARPS = 8;

template <typename T, int V>
struct alignas(sizeof(T) * V) Chunk16 {
    T v[V];
};

// The expert of `row`: the last e with offsets[e] <= row (E: none).
__device__ __forceinline__ int expert_of(const int *offsets, int E, int row) {
    int lo = 0, hi = E + 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (offsets[mid] <= row)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// ROWS of a warp are loaded together.  With enough blocks to fill the GPU several
// times over, one row and more warps do better (8192 x 8192 in bf16: 61 us, four
// rows 120); with few, four (1024 x 1024 in FP32: 5.4 us, one row 7.1).
template <typename T, int V, int ACT, int ROWS>
__global__ void __launch_bounds__(GWARPS * 32)
activation_gradient_kernel(int M, int N, int E, const int *__restrict__ offsets, const T *__restrict__ dy,
                           long long lddy, const T *__restrict__ z, long long ldz, void *__restrict__ dz,
                           long long lddz, float *__restrict__ sums, int strips) {
    constexpr bool F32 = std::is_same<T, float>::value;
    __shared__ float part[GWARPS][32 * V];
    tc::grid_trigger();
    tc::grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunk = blockIdx.x / strips, strip = blockIdx.x - chunk * strips;
    const int col = strip * 32 * V + lane * V;
    const int r1 = min(M, (chunk + 1) * CHUNK);
    int row = chunk * CHUNK;
    while (row < r1) {
        int e = 0, end = r1;
        if (E >= 0) {
            e = expert_of(offsets, E, row);
            if (e < E) end = min(r1, max(offsets[e + 1], row + 1));
        }
        const bool counted = E < 0 || e < E;
        float sum[V];
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] = 0.0f;
        if (counted && col < N)
            for (int r0 = row + warp; r0 < end; r0 += GWARPS * ROWS) {
                Chunk16<T, V> d[ROWS], zz[ROWS];
#pragma unroll
                for (int u = 0; u < ROWS; ++u) {
                    const long long r = r0 + u * GWARPS;
                    if (r < end) {
                        d[u] = *reinterpret_cast<const Chunk16<T, V> *>(dy + r * lddy + col);
                        if constexpr (ACT != LINEAR_ACT_NONE) zz[u] = *reinterpret_cast<const Chunk16<T, V> *>(z + r * ldz + col);
                    }
                }
#pragma unroll
                for (int u = 0; u < ROWS; ++u) {
                    const long long r = r0 + u * GWARPS;
                    if (r >= end) break;
                    float g[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        g[i] = to_f(d[u].v[i]);
                        if constexpr (ACT != LINEAR_ACT_NONE) g[i] *= lt::slope<ACT, F32>(to_f(zz[u].v[i]));
                        sum[i] += g[i];
                    }
                    if (dz == nullptr) continue;
                    if constexpr (F32) {
                        auto *o = static_cast<__nv_bfloat16 *>(dz) + r * lddz + col;
                        const long long piece = static_cast<long long>(M) * lddz;
                        Chunk16<__nv_bfloat16, V> a, b, c;
#pragma unroll
                        for (int i = 0; i < V; ++i) pieces(g[i], a.v[i], b.v[i], c.v[i]);
                        *reinterpret_cast<Chunk16<__nv_bfloat16, V> *>(o) = a;
                        *reinterpret_cast<Chunk16<__nv_bfloat16, V> *>(o + piece) = b;
                        *reinterpret_cast<Chunk16<__nv_bfloat16, V> *>(o + 2 * piece) = c;
                    } else {
                        Chunk16<T, V> a;
#pragma unroll
                        for (int i = 0; i < V; ++i) a.v[i] = from_f<T>(g[i]);
                        *reinterpret_cast<Chunk16<T, V> *>(static_cast<T *>(dz) + r * lddz + col) = a;
                    }
                }
            }
        if (sums != nullptr && counted) {
#pragma unroll
            for (int i = 0; i < V; ++i) part[warp][i * 32 + lane] = sum[i];
            __syncthreads();
            for (int i = threadIdx.x; i < 32 * V; i += GWARPS * 32) {
                const int c = strip * 32 * V + (i & 31) * V + (i >> 5);
                float t = 0.0f;
#pragma unroll
                for (int w = 0; w < GWARPS; ++w) t += part[w][i];
                if (c < N) sums[static_cast<long long>(chunk + (E < 0 ? 0 : e)) * N + c] = t;
            }
            __syncthreads();
        }
        row = end;
    }
}

// Block (32, 8) per 32 columns of an expert: warp y adds chunks y, y + 8, ...
template <typename T>
__global__ void __launch_bounds__(256) column_sums_kernel(int M, int N, int E, const int *__restrict__ offsets,
                                                          const float *__restrict__ sums, T *__restrict__ dbias,
                                                          int strips) {
    __shared__ float part[8][32];
    tc::grid_trigger();
    tc::grid_wait();
    const int e = blockIdx.x / strips, col = (blockIdx.x - e * strips) * 32 + threadIdx.x;
    float t = linear_prep::column_sum(sums, M, N, E, offsets, e, col, threadIdx.y, 8);
    part[threadIdx.y][threadIdx.x] = t;
    __syncthreads();
    if (threadIdx.y == 0 && col < N) {
        t = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += part[i][threadIdx.x];
        dbias[static_cast<long long>(e) * N + col] = from_f<T>(t);
    }
}

template <typename T>
cudaError_t activation_gradient_t(int act, int M, int N, int E, const int *offsets, const void *dy, long long lddy,
                                  const void *z, long long ldz, void *dz, long long lddz, float *sums,
                                  cudaStream_t stream) {
    if (dz == nullptr && sums == nullptr) return cudaSuccess;
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    const bool vec = N % V == 0 && lddy % V == 0 && reinterpret_cast<uintptr_t>(dy) % 16 == 0 &&
                     (act == LINEAR_ACT_NONE || (ldz % V == 0 && reinterpret_cast<uintptr_t>(z) % 16 == 0));
    const int strip = 32 * (vec ? V : 1);
    const int strips = (N + strip - 1) / strip;
    const long long blocks = (static_cast<long long>(M) + CHUNK - 1) / CHUNK * strips;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const unsigned grid = static_cast<unsigned>(blocks);
    cudaError_t err = cudaSuccess;
    auto launch = [&](auto kernel) {
        err = tc::launch(kernel, grid, dim3(GWARPS * 32), 0, stream, M, N, E, offsets, static_cast<const T *>(dy), lddy,
                         static_cast<const T *>(z), ldz, dz, lddz, sums, strips);
    };
    auto pick = [&](auto tag) {
        constexpr int ACT = decltype(tag)::value;
        if (!vec)
            launch(activation_gradient_kernel<T, 1, ACT, 4>);
        else if (blocks < 4 * 152)
            launch(activation_gradient_kernel<T, V, ACT, 4>);
        else
            launch(activation_gradient_kernel<T, V, ACT, 1>);
    };
    switch (act) {
        case LINEAR_ACT_RELU: pick(lt::Int<LINEAR_ACT_RELU>{}); break;
        case LINEAR_ACT_SILU: pick(lt::Int<LINEAR_ACT_SILU>{}); break;
        case LINEAR_ACT_GELU: pick(lt::Int<LINEAR_ACT_GELU>{}); break;
        case LINEAR_ACT_GELU_TANH: pick(lt::Int<LINEAR_ACT_GELU_TANH>{}); break;
        default: pick(lt::Int<LINEAR_ACT_NONE>{}); break;
    }
    return err;
}

template <typename T>
cudaError_t column_sums_t(int M, int N, int E, const int *offsets, const float *sums, void *dbias, cudaStream_t stream) {
    const int strips = (N + 31) / 32;
    const long long blocks = static_cast<long long>(strips) * (E < 0 ? 1 : E);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return tc::launch(column_sums_kernel<T>, static_cast<unsigned>(blocks), dim3(32, 8), 0, stream, M, N, E, offsets, sums,
                      static_cast<T *>(dbias), strips);
}

}  // namespace

namespace linear_prep {

cudaError_t copy_operands(int type, const Copy *copies, int n, cudaStream_t stream) {
    if (n == 0) return cudaSuccess;
    sg_nvtx::Range r("linear: operand copies");
    return type == LINEAR_F32    ? copy_operands_t<float>(copies, n, stream)
           : type == LINEAR_BF16 ? copy_operands_t<__nv_bfloat16>(copies, n, stream)
                                 : copy_operands_t<__half>(copies, n, stream);
}

size_t sums_bytes(int M, int N, int E) {
    return (static_cast<size_t>((static_cast<long long>(M) + CHUNK - 1) / CHUNK) + static_cast<size_t>(E)) *
           static_cast<size_t>(N) * sizeof(float);
}

cudaError_t activation_gradient(int type, int act, int M, int N, int E, const int *offsets, const void *dy,
                                long long lddy, const void *z, long long ldz, void *dz, long long lddz, float *sums,
                                cudaStream_t stream) {
    sg_nvtx::Range r("linear: activation gradient");
    if (type == LINEAR_F32)
        return activation_gradient_t<float>(act, M, N, E, offsets, dy, lddy, z, ldz, dz, lddz, sums, stream);
    if (type == LINEAR_BF16)
        return activation_gradient_t<__nv_bfloat16>(act, M, N, E, offsets, dy, lddy, z, ldz, dz, lddz, sums, stream);
    return activation_gradient_t<__half>(act, M, N, E, offsets, dy, lddy, z, ldz, dz, lddz, sums, stream);
}

cudaError_t column_sums(int type, int M, int N, int E, const int *offsets, const float *sums, void *dbias,
                        cudaStream_t stream) {
    sg_nvtx::Range r("linear: column sums");
    return type == LINEAR_F32    ? column_sums_t<float>(M, N, E, offsets, sums, dbias, stream)
           : type == LINEAR_BF16 ? column_sums_t<__nv_bfloat16>(M, N, E, offsets, sums, dbias, stream)
                                 : column_sums_t<__half>(M, N, E, offsets, sums, dbias, stream);
}

}  // namespace linear_prep
