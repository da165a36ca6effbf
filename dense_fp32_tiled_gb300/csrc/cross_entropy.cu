// cross_entropy.cu -- the softmax cross entropy of a product's rows and its
// gradient (C ABI: include/cross_entropy.h), on product.cuh's kernel with
// epilogues of its own.
//
// The tokens lie on the lanes of tensor memory (they are the kernel's features)
// and the vocabulary along its columns, so a thread sees its token's logits one
// after the other: the running maximum and sum need no exchange between lanes.
//   forward   LOG_SUM over all tiles, then a kernel that joins each token's parts.
//   gradient  per piece of the vocabulary: SOFTMAX_GRADIENT makes dz transposed
//             (vocabulary x tokens); dx += dz.w^T and dw = x^T.dz read it in the
//             order that they need by their operands' descriptors.
// Bound by the tensor cores: 2 M N K operations forward, 6 backward (the logits
// are made again: kept they would be M N values to write and read).
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "cross_entropy.h"
#include "linear_few.cuh"
#include "linear_prep.cuh"
#include "nvtx_range.cuh"
#include "product.cuh"
#include "tensor_core.cuh"

namespace {

using namespace product;

// ---- each token's parts joined ---------------------------------------------------
// A block takes `tokens` tokens (a power of two, up to 32) and gives each as many
// threads: thread k takes parts k, k + threads, ..., four at a time, and the
// threads' results are joined by halves.
constexpr int JOIN_THREADS = 256;
__device__ __forceinline__ float2 join(float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x), ref = m == -INFINITY ? 0.0f : m;
    return make_float2(m, a.y * expf(a.x - ref) + b.y * expf(b.x - ref));
}
__global__ void __launch_bounds__(JOIN_THREADS)
join_kernel(const float2 *__restrict__ parts, int n, int M, int N, int tokens, const Loss l, float *__restrict__ loss,
            float *__restrict__ lse) {
    __shared__ float2 part[JOIN_THREADS];
    const int at = threadIdx.x & (tokens - 1), each = JOIN_THREADS / tokens;
    const int i = blockIdx.x * tokens + at;
    tc::grid_trigger();
    tc::grid_wait();
    const float2 none = make_float2(-INFINITY, 0.0f);
    float2 a = none;
    if (i < M)
        for (int k = threadIdx.x / tokens; k < n; k += 4 * each) {
            float2 p[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) p[u] = k + u * each < n ? parts[static_cast<long long>(k + u * each) * M + i] : none;
            a = join(a, join(join(p[0], p[1]), join(p[2], p[3])));
        }
    part[threadIdx.x] = a;
    for (int k = JOIN_THREADS / 2; k >= tokens; k >>= 1) {
        __syncthreads();
        if (threadIdx.x < k) part[threadIdx.x] = join(part[threadIdx.x], part[threadIdx.x + k]);
    }
    if (threadIdx.x >= tokens || i >= M) return;
    a = part[threadIdx.x];
    const float s = logf(a.y);
    const long long t = target_of(l, i);
    lse[i] = a.x + s;
    // not lse - hit: the rounding of lse is of the logits' size, and where the target is
    // near the largest logit the difference to that is exact and the loss small
    loss[i] = t >= 0 && t < N ? (a.x - l.hit[i]) + s : 0.0f;
}

// ---- few tokens in FP32 ---------------------------------------------------------------
// The product kernel wants the weight in three bf16 pieces, which for few tokens costs
// more than all else (4 x 56678 x 1024: 86 of 154 us); linear's form for few tokens reads
// it once as it is.  It leaves the logits of those few tokens in the workspace,
// and a block here makes a part of STRIP of a token's.
constexpr int STRIP_THREADS = 256, STRIP = 8 * STRIP_THREADS;
__global__ void __launch_bounds__(STRIP_THREADS) strips_kernel(const float *__restrict__ z, int M, int N, int strips, const Loss l) {
    __shared__ float2 part[STRIP_THREADS / 32];
    const int i = blockIdx.x / strips, strip = blockIdx.x - i * strips;
    const int j0 = strip * STRIP;
    const float *row = z + static_cast<long long>(i) * N;
    tc::grid_trigger();
    tc::grid_wait();
    const long long t = target_of(l, i);
    float v[8];
    float2 a = make_float2(-INFINITY, 0.0f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int j = j0 + k * STRIP_THREADS + threadIdx.x;
        v[k] = j < N ? row[j] : -INFINITY;
        a.x = fmaxf(a.x, v[k]);
        if (j < N && j == t) l.hit[i] = v[k];
    }
    const float ref = a.x == -INFINITY ? 0.0f : a.x;
#pragma unroll
    for (int k = 0; k < 8; ++k) a.y += expf(v[k] - ref);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1)
        a = join(a, make_float2(__shfl_xor_sync(0xffffffffu, a.x, k), __shfl_xor_sync(0xffffffffu, a.y, k)));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < STRIP_THREADS / 32; ++w) a = join(a, part[w]);
    l.parts[static_cast<long long>(strip) * M + i] = a;
}

// ---- what the gradient's epilogue needs of each token -------------------------------
// 16-bit types: a and g as fractions of the largest finite one of them (times `up`), and
// alpha, which the products take that back with.  Each block finds the largest by itself.
constexpr int TOKEN_THREADS = 1024;
constexpr int TOKEN_BLOCKS = 152;
__device__ __forceinline__ void gradients_of(const Loss &l, const float *dloss, const float *dlse, int i, int N, float &a, float &g,
                                             int &t) {
    const long long at = target_of(l, i);
    t = at >= 0 && at < N ? static_cast<int>(at) : -1;
    g = t >= 0 && dloss != nullptr ? dloss[i] : 0.0f;
    a = dlse != nullptr ? g + dlse[i] : g;
}
__global__ void __launch_bounds__(TOKEN_THREADS)
tokens_kernel(int M, int N, const Loss l, const float *__restrict__ dloss, const float *__restrict__ dlse,
              const float *__restrict__ lse, int fractions, float up, Token *__restrict__ tokens, float *__restrict__ alpha) {
    __shared__ float most[TOKEN_THREADS / 32];
    tc::grid_trigger();
    tc::grid_wait();
    float scale = 1.0f;
    if (fractions) {
        float m = 0.0f;
        for (int i = threadIdx.x; i < M; i += TOKEN_THREADS) {
            float a, g;
            int t;
            gradients_of(l, dloss, dlse, i, N, a, g, t);
            a = fabsf(a), g = fabsf(g);
            if (a < INFINITY) m = fmaxf(m, a);  // an infinity or a NaN is its token's alone
            if (g < INFINITY) m = fmaxf(m, g);
        }
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
        if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
        __syncthreads();
        for (int k = 0; k < TOKEN_THREADS / 32; ++k) m = fmaxf(m, most[k]);
        scale = m > 0.0f ? m : 1.0f;
        if (blockIdx.x == 0 && threadIdx.x == 0) *alpha = scale / up;
    }
    // unsigned: a step past the last of the most tokens is more than an int holds.  (64 bits took 1 us longer.)
    for (unsigned i = blockIdx.x * TOKEN_THREADS + threadIdx.x; i < static_cast<unsigned>(M); i += gridDim.x * TOKEN_THREADS) {
        Token k;
        gradients_of(l, dloss, dlse, static_cast<int>(i), N, k.a, k.g, k.target);
        k.lse = lse[i];
        if (fractions) {
            k.lse *= lt::kLog2E;
            k.a = k.a / scale * up;
            k.g = k.g / scale * up;
        }
        tokens[i] = k;
    }
}

// ---- host ----------------------------------------------------------------------------
struct Ready {
    int state = 0;
    unsigned long long ctx = 0;
};
std::mutex g_mutex;
Ready g_ready[64];

template <int EPI>
bool opt_in_all() {
    return opt_in<1, __nv_bfloat16, EPI>() && opt_in<2, __nv_bfloat16, EPI>() && opt_in<1, __half, EPI>() && opt_in<2, __half, EPI>() &&
           opt_in<1, float, EPI>() && opt_in<2, float, EPI>();
}
int ready(Device *d) {
    const int st = set_up(d);
    if (st != SGEMM_OK) return st;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return SGEMM_ERR_DEVICE;
    }
    std::lock_guard<std::mutex> lock(g_mutex);
    Ready &r = g_ready[dev];
    if (r.state == 0 || r.ctx != d->ctx) {
        r.ctx = d->ctx;
        const bool many = opt_in<1, __nv_bfloat16, SOFTMAX_GRADIENT, true>() && opt_in<2, __nv_bfloat16, SOFTMAX_GRADIENT, true>() &&
                          opt_in<1, __half, SOFTMAX_GRADIENT, true>() && opt_in<2, __half, SOFTMAX_GRADIENT, true>();
        r.state = opt_in_all<LOG_SUM>() && opt_in_all<SOFTMAX_GRADIENT>() && many && opt_in_all<SCALED_SUM>() ? 1 : -1;
        (void)cudaGetLastError();
    }
    return r.state > 0 ? SGEMM_OK : SGEMM_ERR_DEVICE;
}

struct Head {
    int type, M, N, K;
    const void *x, *w, *targets;
    long long ldx, ldw;
    int w_order, target_bytes;
};
int check_sizes(const Head &h) {
    if (h.type < LINEAR_F32 || h.type > LINEAR_F16 || (h.w_order != 0 && h.w_order != 1)) return SGEMM_ERR_INVALID_ARG;
    if (h.M < 0 || h.N < 0 || h.K < 0) return SGEMM_ERR_INVALID_DIM;
    if (h.M > INT_MAX - 1024 || h.N > INT_MAX - 1024 || h.K > INT_MAX - 1024) return SGEMM_ERR_INVALID_DIM;
    return SGEMM_OK;
}
long long w_inner(const Head &h) { return h.w_order ? h.K : h.N; }
long long w_outer(const Head &h) { return h.w_order ? h.N : h.K; }
int check(const Head &h) {
    const int st = check_sizes(h);
    if (st != SGEMM_OK) return st;
    if (h.target_bytes != 4 && h.target_bytes != 8) return SGEMM_ERR_INVALID_ARG;
    if (h.ldx < at_least_1(h.K) || h.ldw < at_least_1(w_inner(h))) return SGEMM_ERR_INVALID_LD;
    return SGEMM_OK;
}
Matrix x_matrix(const Head &h) { return row_matrix(h.x, h.M, h.K, h.ldx); }
Matrix w_matrix(const Head &h) {
    Matrix m;
    m.base = h.w;
    m.inner = w_inner(h);
    m.outer = w_outer(h);
    m.ld = h.ldw;
    m.plane = m.outer * h.ldw;
    return m;
}
Span w_span(const void *p, const Head &h, long long ld) { return span(p, w_outer(h), w_inner(h), ld, lt::type_bytes(h.type)); }

// ---- forward -------------------------------------------------------------------------
linear_few::Few few(const Head &h) {
    linear_few::Few p;
    memset(&p, 0, sizeof p);
    p.T = h.M, p.F = h.N, p.K = h.K, p.x = h.x, p.w = h.w, p.ldx = h.ldx, p.ldw = h.ldw, p.ldo = h.N, p.order = h.w_order;
    return p;
}
bool few_tokens(const Head &h) { return h.type == LINEAR_F32 && h.K > 0 && linear_few::takes(h.type, few(h)); }

struct ForwardBytes {
    size_t parts, hit, z, total;
};
ForwardBytes forward_bytes(const Head &h) {
    ForwardBytes b{};
    if (check_sizes(h) != SGEMM_OK || h.M == 0 || h.N == 0) return b;
    const long long columns = log_sum_columns(h.N, h.M), tiles = (h.N + columns - 1) / columns;
    b.parts = up256(2 * tiles * h.M * static_cast<long long>(sizeof(float2)));
    b.hit = up256(4LL * h.M);
    if (few_tokens(h)) b.z = up256(4LL * h.M * h.N);
    b.total = b.parts + b.hit + b.z;
    if (h.K > 0 && b.z == 0) b.total += operand_bytes(h.type, x_matrix(h)) + operand_bytes(h.type, w_matrix(h));
    return b;
}

int forward(const Head &h, float *loss, float *lse, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    int st = check(h);
    if (st != SGEMM_OK) return st;
    if (h.M == 0) return SGEMM_OK;
    if (loss == nullptr || lse == nullptr || h.targets == nullptr || (h.K > 0 && h.N > 0 && (h.x == nullptr || h.w == nullptr)))
        return SGEMM_ERR_NULL_PTR;
    const ForwardBytes need = forward_bytes(h);
    if (need.total > 0 && workspace == nullptr) return SGEMM_ERR_NULL_PTR;
    const int b = lt::type_bytes(h.type);
    if (misaligned(h.x, b) || misaligned(h.w, b) || misaligned(h.targets, h.target_bytes) || misaligned(loss, 4) ||
        misaligned(lse, 4) || misaligned(workspace, 256) || workspace_bytes < need.total)
        return SGEMM_ERR_INVALID_ARG;
    const Span out[3] = {span(loss, 1, h.M, h.M, 4), span(lse, 1, h.M, h.M, 4),
                         span(workspace, 1, static_cast<long long>(need.total), static_cast<long long>(need.total), 1)};
    const Span in[3] = {span(h.x, h.M, h.K, h.ldx, b), w_span(h.w, h, h.ldw), span(h.targets, 1, h.M, h.M, h.target_bytes)};
    for (int i = 0; i < 3; ++i) {
        for (const Span &s : in)
            if (overlap(out[i], s)) return SGEMM_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return SGEMM_ERR_ALIAS;
    }
    Device d;
    st = ready(&d);
    if (st != SGEMM_OK) return st;
    char *ws = static_cast<char *>(workspace);
    Product p;
    memset(&p, 0, sizeof p);
    p.loss.parts = reinterpret_cast<float2 *>(ws);
    p.loss.hit = reinterpret_cast<float *>(ws + need.parts);
    p.loss.targets = h.targets;
    p.loss.target_bytes = h.target_bytes;
    int parts = 0;
    auto failed = [] {
        (void)cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    };
    if (need.z > 0) {
        linear_few::Few f = few(h);
        f.out = ws + need.parts + need.hit;
        f.sms = d.sms;
        if (linear_few::run(h.type, f, stream) != cudaSuccess) return failed();
        parts = (h.N + STRIP - 1) / STRIP;
        sg_nvtx::Range r("cross entropy: strips");
        if (tc::launch(strips_kernel, static_cast<unsigned>(parts) * h.M, dim3(STRIP_THREADS), 0, stream, static_cast<const float *>(f.out),
                       h.M, h.N, parts, p.loss) != cudaSuccess)
            return failed();
    } else if (h.N > 0) {
        Operand P, Q;
        if (h.K > 0) {
            Copies copies(ws + need.parts + need.hit);
            P = copies.operand(h.type, x_matrix(h), false);
            Q = copies.operand(h.type, w_matrix(h), h.w_order == 0);
            st = copies.run(h.type, stream);
            if (st != SGEMM_OK) return st;
        }
        p.T = h.N;
        p.F = h.M;
        p.K = h.K;
        p.mode = DENSE;
        st = run_product<LOG_SUM>(h.type, p, P, Q, d, stream, &parts);
        if (st != SGEMM_OK) return st;
        parts *= 2;
    }
    sg_nvtx::Range r("cross entropy: join");
    int tokens = 32;  // of a block: fewer where there are few
    while (tokens > 1 && h.M < tokens * 2 * d.sms) tokens /= 2;
    const cudaError_t err = tc::launch(join_kernel, static_cast<unsigned>((static_cast<long long>(h.M) + tokens - 1) / tokens),
                                       dim3(JOIN_THREADS), 0, stream, static_cast<const float2 *>(p.loss.parts), parts, h.M, h.N, tokens,
                                       p.loss, loss, lse);
    return err == cudaSuccess ? SGEMM_OK : failed();
}

// ---- gradient ------------------------------------------------------------------------
constexpr int SMS = 152, MOST_CHUNKS = 64;

// dx (M rows of K) from the sums of its chunks, in their order: a block takes 256 of a row.
template <typename T>
__global__ void __launch_bounds__(256) chunks_kernel(const float *__restrict__ acc, int chunks, int M, int K, int strips,
                                                     const float *alpha, T *__restrict__ dx, long long lddx) {
    tc::grid_trigger();
    tc::grid_wait();
    const int row = blockIdx.x / strips, k = (blockIdx.x - row * strips) * 256 + threadIdx.x;
    if (k >= K) return;
    const long long all = static_cast<long long>(M) * K;
    const float *from = acc + static_cast<long long>(row) * K + k;
    float s = 0.0f;
#pragma unroll 8
    for (int c = 0; c < chunks; ++c) s += from[c * all];
    dx[row * lddx + k] = from_f<T>(alpha != nullptr ? s * *alpha : s);
}

struct BackwardBytes {
    int piece;   // columns of the vocabulary at a time
    int chunks;  // of them, most sums of dx side by side
    size_t dz, tokens, acc, total;
};
BackwardBytes backward_bytes(const Head &h, bool want_dx, bool want_dw) {
    BackwardBytes b{};
    if (check_sizes(h) != SGEMM_OK || h.M == 0 || h.N == 0 || h.K == 0 || (!want_dx && !want_dw)) return b;
    // as few pieces as the room allows, of the same size, of whole tiles
    const long long most = at_least_1(CROSS_ENTROPY_PIECE / up8(h.M) / 256) * 256;
    const long long pieces = (h.N + most - 1) / most;
    const long long piece = ((h.N + pieces - 1) / pieces + 255) / 256 * 256;
    b.piece = static_cast<int>(piece < h.N ? piece : h.N);
    b.dz = up256(b.piece * up8(h.M) * 2 * (h.type == LINEAR_F32 ? 3 : 1));
    b.tokens = up256(static_cast<long long>(sizeof(Token)) * h.M) + 256;
    // where dx has fewer tiles than there are SMs, the vocabulary is shared out
    const long long tiles = ((h.M + 127LL) / 128) * ((h.K + 127LL) / 128);
    b.chunks = tiles > SMS / 2 ? 1 : static_cast<int>(SMS / tiles < MOST_CHUNKS ? SMS / tiles : MOST_CHUNKS);
    b.acc = want_dx && (b.piece < h.N || b.chunks > 1) ? up256(4LL * b.chunks * h.M * h.K) : 0;
    b.total = b.dz + b.tokens + b.acc + operand_bytes(h.type, x_matrix(h)) + operand_bytes(h.type, w_matrix(h));
    return b;
}
// Columns begin .. begin + n of the vocabulary of an operand that holds the weight.
Operand columns(Operand w, int w_order, int begin, int n) {
    w.base = static_cast<const char *>(w.base) + 2 * (w_order ? begin * w.ld : begin);
    (w_order ? w.outer : w.inner) = n;
    return w;
}

int backward(const Head &h, const float *dloss, const float *dlse, const float *lse, void *dx, long long lddx, void *dw, long long lddw,
             void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    int st = check(h);
    if (st != SGEMM_OK) return st;
    if ((dx != nullptr && lddx < at_least_1(h.K)) || (dw != nullptr && lddw < at_least_1(w_inner(h)))) return SGEMM_ERR_INVALID_LD;
    if ((dx == nullptr && dw == nullptr) || h.K == 0) return SGEMM_OK;
    const bool empty = h.M == 0 || h.N == 0;
    if (!empty && (h.x == nullptr || h.w == nullptr || h.targets == nullptr || lse == nullptr)) return SGEMM_ERR_NULL_PTR;
    const BackwardBytes need = backward_bytes(h, dx != nullptr, dw != nullptr);
    if (need.total > 0 && workspace == nullptr) return SGEMM_ERR_NULL_PTR;
    const int b = lt::type_bytes(h.type);
    if (misaligned(h.x, b) || misaligned(h.w, b) || misaligned(h.targets, h.target_bytes) || misaligned(dloss, 4) ||
        misaligned(dlse, 4) || misaligned(lse, 4) || misaligned(dx, b) || misaligned(dw, b) || misaligned(workspace, 256) ||
        workspace_bytes < need.total)
        return SGEMM_ERR_INVALID_ARG;
    const Span out[3] = {span(dx, h.M, h.K, lddx, b), w_span(dw, h, lddw),
                         span(workspace, 1, static_cast<long long>(need.total), static_cast<long long>(need.total), 1)};
    const Span in[6] = {span(h.x, h.M, h.K, h.ldx, b), w_span(h.w, h, h.ldw), span(h.targets, 1, h.M, h.M, h.target_bytes),
                        span(dloss, 1, h.M, h.M, 4), span(dlse, 1, h.M, h.M, 4), span(lse, 1, h.M, h.M, 4)};
    for (int i = 0; i < 3; ++i) {
        for (const Span &s : in)
            if (overlap(out[i], s)) return SGEMM_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return SGEMM_ERR_ALIAS;
    }
    if (empty) {
        cudaError_t err = cudaSuccess;
        if (dx != nullptr && h.M > 0)
            err = cudaMemset2DAsync(dx, static_cast<size_t>(lddx) * b, 0, static_cast<size_t>(h.K) * b, static_cast<size_t>(h.M), stream);
        if (err == cudaSuccess && dw != nullptr && h.N > 0)
            err = cudaMemset2DAsync(dw, static_cast<size_t>(lddw) * b, 0, static_cast<size_t>(w_inner(h)) * b,
                                    static_cast<size_t>(w_outer(h)), stream);
        if (err == cudaSuccess) return SGEMM_OK;
        (void)cudaGetLastError();
        return SGEMM_ERR_LAUNCH;
    }
    Device d;
    st = ready(&d);
    if (st != SGEMM_OK) return st;
    const bool f32 = h.type == LINEAR_F32;
    char *ws = static_cast<char *>(workspace);
    Token *tokens = reinterpret_cast<Token *>(ws + need.dz);
    float *alpha = reinterpret_cast<float *>(ws + need.dz + need.tokens - 256);
    Copies copies(ws + need.dz + need.tokens + need.acc);
    const Operand X = copies.operand(h.type, x_matrix(h), false);
    const Operand W = copies.operand(h.type, w_matrix(h), h.w_order == 0);
    st = copies.run(h.type, stream);
    if (st != SGEMM_OK) return st;
    Product p;
    memset(&p, 0, sizeof p);
    p.mode = DENSE;
    p.loss.targets = h.targets;
    p.loss.target_bytes = h.target_bytes;
    {
        sg_nvtx::Range r("cross entropy: tokens");
        const int blocks = (h.M + TOKEN_THREADS - 1) / TOKEN_THREADS;
        if (tc::launch(tokens_kernel, static_cast<unsigned>(blocks < TOKEN_BLOCKS ? blocks : TOKEN_BLOCKS), dim3(TOKEN_THREADS), 0, stream,
                       h.M, h.N, p.loss, dloss, dlse, lse, f32 ? 0 : 1, h.type == LINEAR_F16 ? 16384.0f : 1.0f, tokens,
                       alpha) != cudaSuccess) {
            (void)cudaGetLastError();
            return SGEMM_ERR_LAUNCH;
        }
    }
    p.loss.tokens = tokens;
    p.loss.alpha = f32 ? nullptr : alpha;
    p.loss.acc = reinterpret_cast<float *>(ws + need.dz + need.tokens);
    const long long ldz = up8(h.M);
    int chunks = -need.chunks;
    // 64 bits: pieces are whole tiles, so past the last one of the largest N lies more than an int holds
    for (long long next = 0; next < h.N; next += need.piece) {
        const int begin = static_cast<int>(next), n = h.N - begin < need.piece ? h.N - begin : need.piece;
        Operand Z;  // n rows of M
        Z.base = ws;
        Z.inner = h.M;
        Z.outer = n;
        Z.ld = ldz;
        Z.plane = n * ldz;
        Z.planes = f32 ? PIECES : 1;
        const Operand Wn = columns(W, h.w_order, begin, n);
        Product z = p;
        z.T = n;
        z.F = h.M;
        z.K = h.K;
        z.out = ws;
        z.ldo = ldz;
        z.loss.begin = begin;
        z.loss.piece = Z.plane;
        st = run_product<SOFTMAX_GRADIENT>(h.type, z, X, Wn, d, stream);
        if (st != SGEMM_OK) return st;
        const bool two = dx != nullptr && dw != nullptr;
        if (dx != nullptr) {
            Product g = p;
            Operand P = Wn, Q = Z;
            P.mn = h.w_order == 1;
            Q.mn = true;
            g.T = h.M;
            g.F = h.K;
            g.K = n;
            g.out = dx;
            g.ldo = lddx;
            g.order = two ? ORDER_FIRST : ORDER_ALONE;
            g.loss.first = begin == 0;
            g.loss.last = begin + n == h.N;
            const bool whole = need.piece == h.N;
            if (f32 && whole && need.chunks == 1)
                st = run_layer(h.type, g, P, Q, d, stream);
            else
                st = run_product<SCALED_SUM>(h.type, g, P, Q, d, stream, nullptr, &chunks);
            if (st != SGEMM_OK) return st;
        }
        if (dw != nullptr) {
            Product g = p;
            Operand Xt = X, Zk = Z;
            Xt.mn = true;
            Zk.mn = false;
            // rows of dw in memory: K of N (order 0) or N of K (order 1)
            g.T = h.w_order ? n : h.K;
            g.F = h.w_order ? h.K : n;
            g.K = h.M;
            g.out = static_cast<char *>(dw) + b * (h.w_order ? begin * lddw : begin);
            g.ldo = lddw;
            g.order = two ? ORDER_BESIDE : ORDER_ALONE;
            g.loss.first = g.loss.last = 1;
            g.loss.acc = nullptr;
            const Operand &P = h.w_order ? Xt : Zk, &Q = h.w_order ? Zk : Xt;
            st = f32 ? run_layer(h.type, g, P, Q, d, stream) : run_product<SCALED_SUM>(h.type, g, P, Q, d, stream);
            if (st != SGEMM_OK) return st;
        }
    }
    if (dx != nullptr && chunks > 1) {
        sg_nvtx::Range r("cross entropy: sum of chunks");
        const int strips = (h.K + 255) / 256;  // chunks are for few tiles: M * strips fits
        auto sum = [&](auto el) {
            using El = decltype(el);
            return tc::launch(chunks_kernel<El>, static_cast<unsigned>(h.M) * strips, dim3(256), 0, stream,
                              static_cast<const float *>(p.loss.acc), chunks, h.M, h.K, strips, p.loss.alpha, static_cast<El *>(dx), lddx);
        };
        const cudaError_t err = f32 ? sum(float()) : h.type == LINEAR_BF16 ? sum(__nv_bfloat16()) : sum(__half());
        if (err != cudaSuccess) {
            (void)cudaGetLastError();
            return SGEMM_ERR_LAUNCH;
        }
    }
    return SGEMM_OK;
}

Head head(int type, int M, int N, int K, const void *x, long long ldx, const void *w, long long ldw, int w_order, const void *targets,
          int target_bytes) {
    Head h{};
    h.type = type, h.M = M, h.N = N, h.K = K, h.x = x, h.w = w, h.targets = targets, h.ldx = ldx, h.ldw = ldw, h.w_order = w_order;
    h.target_bytes = target_bytes;
    return h;
}

}  // namespace

extern "C" int linear_cross_entropy_forward(int type, int M, int N, int K, const void *x, int64_t ldx, const void *w, int64_t ldw,
                                            int w_order, const void *targets, int target_bytes, float *loss, float *lse,
                                            void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    return forward(head(type, M, N, K, x, ldx, w, ldw, w_order, targets, target_bytes), loss, lse, workspace, workspace_bytes, stream);
}

extern "C" size_t linear_cross_entropy_forward_workspace_size(int type, int M, int N, int K, const void *x, int64_t ldx,
                                                              const void *w, int64_t ldw, int w_order) {
    return forward_bytes(head(type, M, N, K, x, ldx, w, ldw, w_order, nullptr, 4)).total;
}

extern "C" int linear_cross_entropy_backward(int type, int M, int N, int K, const float *dloss, const float *dlse, const void *x,
                                             int64_t ldx, const void *w, int64_t ldw, int w_order, const void *targets,
                                             int target_bytes, const float *lse, void *dx, int64_t lddx, void *dw, int64_t lddw,
                                             void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    return backward(head(type, M, N, K, x, ldx, w, ldw, w_order, targets, target_bytes), dloss, dlse, lse, dx, lddx, dw, lddw, workspace,
                    workspace_bytes, stream);
}

extern "C" size_t linear_cross_entropy_backward_workspace_size(int type, int M, int N, int K, const void *x, int64_t ldx,
                                                               const void *w, int64_t ldw, int w_order, int want_dx, int want_dw) {
    return backward_bytes(head(type, M, N, K, x, ldx, w, ldw, w_order, nullptr, 4), want_dx != 0, want_dw != 0).total;
}
