// linear.cu -- the layer products of GB300 (sm_103a): y = act(x.w + bias) +
// residual, the same over rows grouped by expert, and the products of their
// gradients, all on product.cuh's kernel (C ABI: include/linear.h).
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "ctx_key.cuh"
#include "linear.h"
#include "linear_few.cuh"
#include "linear_prep.cuh"
#include "product.cuh"

namespace {

using namespace product;

__device__ unsigned g_linear_timeout;

std::mutex g_mutex;
Device g_devices[64];

}  // namespace

namespace product {

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
            minor != 3 || d.sms < 2 || encode_fn() == nullptr || !opt_in<1, float, LAYER>() || !opt_in<2, float, LAYER>() ||
            !opt_in<1, __nv_bfloat16, LAYER>() || !opt_in<2, __nv_bfloat16, LAYER>() || !opt_in<1, __half, LAYER>() ||
            !opt_in<2, __half, LAYER>() ||
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

int run_layer(int type, const Product &p, const Operand &P, const Operand &Q, const Device &d, cudaStream_t stream) {
    return run_product<LAYER>(type, p, P, Q, d, stream);
}

}  // namespace product

namespace {

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
    return run_layer(c.type, p, P, Q, d, c.stream);
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
        st = run_layer(c.type, p, P_dx, Q, d, c.stream);
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
        st = run_layer(c.type, p, c.w_order ? X : Z, c.w_order ? Z : X, d, c.stream);
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
