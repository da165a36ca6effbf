/* fast_call.c -- the common calls of _layers.py without the interpreter.
 *
 * A decoding step's product takes some microseconds on the GPU, and marshalling
 * it in Python takes longer than that (14 us a call; 7 through here).  Each
 * function below does what its namesake in _layers.py does for a call on the
 * current device and stream whose arguments are as they should be, and returns
 * NotImplemented for anything else: another device or a strange argument goes
 * through _layers.py, which serves or refuses it.  The arithmetic, the checks
 * of sizes and the status codes are the library's, whose functions it calls by
 * the addresses that bind() gets.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stddef.h>
#include <stdint.h>

typedef void *stream_t;
static struct {
    int (*linear_forward)(int, int, int, int, const void *, int64_t, const void *, int64_t, int, const void *, const void *,
                          int64_t, int, void *, int64_t, void *, int64_t, void *, size_t, stream_t);
    size_t (*linear_forward_workspace_size)(int, int, int, int, const void *, int64_t, const void *, int64_t, int);
    int (*expert_linear_forward)(int, int, int, int, int, const int *, const void *, int64_t, const void *, int64_t, int64_t,
                                 int, const void *, const void *, int64_t, int, void *, int64_t, void *, int64_t, void *,
                                 size_t, stream_t);
    size_t (*expert_linear_forward_workspace_size)(int, int, int, int, int, const void *, int64_t, const void *, int64_t,
                                                   int64_t, int);
    int (*linear_backward)(int, int, int, int, const void *, int64_t, const void *, int64_t, const void *, int64_t, int,
                           const void *, int64_t, int, void *, int64_t, void *, int64_t, void *, void *, size_t, stream_t);
    size_t (*linear_backward_workspace_size)(int, int, int, int, const void *, int64_t, const void *, int64_t, const void *,
                                             int64_t, int, int, int, int, int);
    int (*expert_linear_backward)(int, int, int, int, int, const int *, const void *, int64_t, const void *, int64_t,
                                  const void *, int64_t, int64_t, int, const void *, int64_t, int, void *, int64_t, void *,
                                  int64_t, int64_t, void *, void *, size_t, stream_t);
    size_t (*expert_linear_backward_workspace_size)(int, int, int, int, int, const void *, int64_t, const void *, int64_t,
                                                    const void *, int64_t, int64_t, int, int, int, int, int);
    int (*expert_sort)(int, int, int, const void *, int, int *, int *, void *, size_t, stream_t);
    size_t (*expert_sort_workspace_size)(int, int, int);
    int (*expert_gather)(int, int, int, int, int, const int *, const int *, const void *, int64_t, void *, int64_t, stream_t);
    int (*expert_combine)(int, int, int, int, const int *, const float *, const void *, int64_t, const void *, int64_t, void *,
                          int64_t, stream_t);
    int (*expert_combine_backward)(int, int, int, int, int, const int *, const int *, const float *, const void *, int64_t,
                                   const void *, int64_t, void *, int64_t, float *, stream_t);
} lib;
static const char *const lib_names[] = {"linear_forward", "linear_forward_workspace_size", "expert_linear_forward",
                                        "expert_linear_forward_workspace_size", "linear_backward",
                                        "linear_backward_workspace_size", "expert_linear_backward",
                                        "expert_linear_backward_workspace_size", "expert_sort", "expert_sort_workspace_size",
                                        "expert_gather", "expert_combine", "expert_combine_backward"};

/* The operators around the layers, bound by bind_more(). */
static struct {
    int (*layer_norm_forward)(int, int, int, const void *, int64_t, const void *, const void *, float, float *, void *, int64_t,
                              stream_t);
    int (*layer_norm_backward)(int, int, int, const void *, int64_t, const void *, int64_t, const void *, const float *, void *,
                               int64_t, void *, void *, void *, size_t, stream_t);
    size_t (*layer_norm_backward_workspace_size)(int, int, int, int);
    int (*expert_choose)(int, int, int, int, const void *, int64_t, const float *, int, int, int, int, int, float, int *, float *,
                         stream_t);
    int (*expert_choose_backward)(int, int, int, int, const float *, const int *, const void *, int64_t, int, int, float, void *,
                                  int64_t, stream_t);
    int (*linear_cross_entropy_forward)(int, int, int, int, const void *, int64_t, const void *, int64_t, int, const void *, int,
                                        float *, float *, void *, size_t, stream_t);
    size_t (*linear_cross_entropy_forward_workspace_size)(int, int, int, int, const void *, int64_t, const void *, int64_t, int);
    int (*linear_cross_entropy_backward)(int, int, int, int, const float *, const float *, const void *, int64_t, const void *,
                                         int64_t, int, const void *, int, const float *, void *, int64_t, void *, int64_t, void *,
                                         size_t, stream_t);
    size_t (*linear_cross_entropy_backward_workspace_size)(int, int, int, int, const void *, int64_t, const void *, int64_t, int,
                                                           int, int);
} more;
static const char *const more_names[] = {"layer_norm_forward", "layer_norm_backward", "layer_norm_backward_workspace_size",
                                         "expert_choose", "expert_choose_backward", "linear_cross_entropy_forward",
                                         "linear_cross_entropy_forward_workspace_size", "linear_cross_entropy_backward",
                                         "linear_cross_entropy_backward_workspace_size"};
static PyObject *scorings; /* NULL: not bound */

/* A launch may wait for room in the stream's queue, and what it waits for, such as a
 * function on the host, may want the interpreter: it is not held meanwhile. */
#define LAUNCH(status, call)   \
    do {                       \
        Py_BEGIN_ALLOW_THREADS \
        status = call;         \
        Py_END_ALLOW_THREADS   \
    } while (0)

/* What bind() keeps: torch's own objects, for the life of the process. */
static PyObject *tensor_type, *empty, *raw_stream, *get_device, *activations, *kinds[3], *int32_type, *int64_type, *uint8_type;
static PyObject *s_dtype, *s_device, *s_shape, *s_stride, *s_data_ptr, *s_get_device, *s_transpose;
static PyObject *empty_names, *minus1, *minus2;

#define UNUSUAL() return PyErr_Occurred() ? (PyErr_Clear(), Py_NewRef(Py_NotImplemented)) : Py_NewRef(Py_NotImplemented)

static int whole(PyObject *o, int64_t *v) { /* 1: *v holds it */
    if (o == NULL) return 0;
    *v = PyLong_AsLongLong(o);
    return !(*v == -1 && PyErr_Occurred());
}
static int64_t call_whole(PyObject *t, PyObject *name, int64_t bad) {
    PyObject *r = PyObject_CallMethodNoArgs(t, name);
    int64_t v;
    const int ok = whole(r, &v);
    Py_XDECREF(r);
    return ok ? v : bad;
}
/* The tuple's numbers, at most three; how many there are, or -1. */
static int numbers(PyObject *tuple, int64_t *v) {
    if (tuple == NULL || !PyTuple_Check(tuple)) return -1;
    const Py_ssize_t n = PyTuple_GET_SIZE(tuple);
    if (n > 3) return -1;
    for (Py_ssize_t i = 0; i < n; ++i)
        if (!whole(PyTuple_GET_ITEM(tuple, i), v + i)) return -1;
    return (int)n;
}

typedef struct {
    int dims;
    int64_t size[3], stride[3];
    void *data;
} Tensor;
/* Shape, strides and address of a tensor of this type on this device; 0 for anything else. */
static int look(PyObject *t, PyObject *dtype, int64_t device, Tensor *out) {
    if (!PyObject_TypeCheck(t, (PyTypeObject *)tensor_type)) return 0;
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    Py_XDECREF(d); /* torch holds its types */
    if (d != dtype || call_whole(t, s_get_device, -1) != device) return 0;
    PyObject *p = PyObject_GetAttr(t, s_shape);
    out->dims = numbers(p, out->size);
    Py_XDECREF(p);
    if (out->dims < 0) return 0;
    p = PyObject_CallMethodNoArgs(t, s_stride);
    const int n = numbers(p, out->stride);
    Py_XDECREF(p);
    if (n != out->dims) return 0;
    out->data = (void *)(intptr_t)call_whole(t, s_data_ptr, -1);
    return out->data != (void *)(intptr_t)-1;
}
static int kind_of(PyObject *t, PyObject **dtype) {
    if (!PyObject_TypeCheck(t, (PyTypeObject *)tensor_type)) return -1;
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    Py_XDECREF(d);
    *dtype = d;
    for (int i = 0; i < 3; ++i)
        if (d == kinds[i]) return i;
    return -1;
}
/* A row-major rows x cols matrix. */
static int rows_of(const Tensor *t, int64_t rows, int64_t cols, int64_t *ld) {
    if (t->dims != 2 || t->size[0] != rows || t->size[1] != cols) return 0;
    if (cols > 1 && t->stride[1] != 1) return 0;
    *ld = t->stride[0];
    if (*ld < cols || *ld < 1) {
        if (rows > 1) return 0;
        *ld = cols > 1 ? cols : 1;
    }
    return 1;
}
static int flat(const Tensor *t, int dims, int64_t a, int64_t b) { /* contiguous, of shape (a,) or (a, b) */
    if (t->dims != dims || t->size[0] != a) return 0;
    if (dims == 1) return t->stride[0] == 1 || a <= 1;
    return t->size[1] == b && (t->stride[1] == 1 || b <= 1) && (t->stride[0] == b || a <= 1);
}
typedef struct {
    int64_t K, N, ld, expert;
    int order;
} Weight;
static int weight_of(const Tensor *t, int dims, Weight *w) {
    if (t->dims != dims) return 0;
    const int64_t K = w->K = t->size[dims - 2], N = w->N = t->size[dims - 1], sk = t->stride[dims - 2],
                  sn = t->stride[dims - 1];
    if (K < 2 || N < 2) return 0; /* strides that mean nothing: the long way */
    w->expert = dims == 3 && t->size[0] > 1 ? t->stride[0] : 0;
    w->order = !(sn == 1 && sk >= N);
    w->ld = w->order ? sn : sk;
    return !w->order || (sk == 1 && sn >= K);
}
static int small(int64_t a, int64_t b, int64_t c) { return a <= INT32_MAX && b <= INT32_MAX && c <= INT32_MAX; }

/* The current device's number and its current stream; 0 if the tensor is not on it. */
static int here(PyObject *t, int64_t *device, stream_t *stream) {
    *device = call_whole(t, s_get_device, -1);
    if (*device < 0) return 0;
    PyObject *r = PyObject_CallNoArgs(get_device);
    int64_t current;
    int ok = whole(r, &current);
    Py_XDECREF(r);
    if (!ok || current != *device) return 0;
    PyObject *n = PyLong_FromLongLong(*device);
    r = n == NULL ? NULL : PyObject_CallOneArg(raw_stream, n);
    Py_XDECREF(n);
    int64_t s = 0;
    ok = whole(r, &s);
    Py_XDECREF(r);
    *stream = (stream_t)(intptr_t)s;
    return ok;
}
/* torch.empty(sizes, dtype=dtype, device=like.device), and its address. */
static PyObject *new_tensor(int dims, const int64_t *size, PyObject *dtype, PyObject *like, void **data) {
    PyObject *shape = PyTuple_New(dims), *r = NULL;
    if (shape == NULL) return NULL;
    for (int i = 0; i < dims; ++i) {
        PyObject *n = PyLong_FromLongLong(size[i]);
        if (n == NULL) goto done;
        PyTuple_SET_ITEM(shape, i, n);
    }
    PyObject *device = PyObject_GetAttr(like, s_device);
    if (device == NULL) goto done;
    PyObject *args[3] = {shape, dtype, device};
    r = PyObject_Vectorcall(empty, args, 1, empty_names);
    Py_DECREF(device);
    if (r != NULL) {
        const int64_t p = call_whole(r, s_data_ptr, -1);
        if (p == -1) Py_CLEAR(r);
        *data = (void *)(intptr_t)p;
    }
done:
    Py_DECREF(shape);
    return r;
}
/* Scratch of this call alone (*hold, to be let go after the launches; NULL: none needed). */
static int scratch(size_t bytes, PyObject *like, PyObject **hold, void **data) {
    *hold = NULL;
    *data = NULL;
    if (bytes == 0) return 1;
    const int64_t size[1] = {(int64_t)bytes};
    *hold = new_tensor(1, size, uint8_type, like, data);
    return *hold != NULL;
}
static int activation(PyObject *name, int *act) {
    PyObject *v = PyDict_GetItemWithError(activations, name);
    int64_t n;
    if (!whole(v, &n)) return 0;
    *act = (int)n;
    return 1;
}

/* forward(x, w, offsets, bias, residual, activation, preact, out) -> out */
static PyObject *forward(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    PyObject *dtype;
    int64_t device, ldr = 0, ldz = 0, ldy;
    stream_t stream;
    int act;
    Tensor x, w, t;
    Weight m;
    const void *bias = NULL, *residual = NULL;
    void *z = NULL, *y, *ws = NULL;
    if (n != 8) UNUSUAL();
    const int kind = kind_of(a[0], &dtype);
    if (kind < 0 || !here(a[0], &device, &stream) || !look(a[0], dtype, device, &x) || !look(a[1], dtype, device, &w) ||
        !activation(a[5], &act))
        UNUSUAL();
    const int grouped = a[2] != Py_None;
    int64_t ldx;
    if (x.dims != 2 || !weight_of(&w, 2 + grouped, &m) || !rows_of(&x, x.size[0], m.K, &ldx)) UNUSUAL();
    const int64_t M = x.size[0], K = m.K, N = m.N, E = grouped ? w.size[0] : 0;
    const int *offsets = NULL;
    if (!small(M, N, K) || E > INT32_MAX) UNUSUAL();
    if (grouped) {
        if (!look(a[2], int32_type, device, &t) || !flat(&t, 1, E + 1, 0)) UNUSUAL();
        offsets = t.data;
    }
    if (a[3] != Py_None) {
        if (!look(a[3], dtype, device, &t) || !(grouped ? flat(&t, 2, E, N) : flat(&t, 1, N, 0))) UNUSUAL();
        bias = t.data;
    }
    if (a[4] != Py_None) {
        if (!look(a[4], dtype, device, &t) || !rows_of(&t, M, N, &ldr)) UNUSUAL();
        residual = t.data;
    }
    if (a[6] != Py_None) {
        if (!look(a[6], dtype, device, &t) || !rows_of(&t, M, N, &ldz)) UNUSUAL();
        z = t.data;
    }
    const size_t need = grouped ? lib.expert_linear_forward_workspace_size(kind, (int)M, (int)N, (int)K, (int)E, x.data, ldx,
                                                                           w.data, m.ld, m.expert, m.order)
                                : lib.linear_forward_workspace_size(kind, (int)M, (int)N, (int)K, x.data, ldx, w.data, m.ld,
                                                                    m.order);
    PyObject *out = a[7], *hold;
    if (out == Py_None) {
        const int64_t size[2] = {M, N};
        out = new_tensor(2, size, dtype, a[0], &y);
        if (out == NULL) UNUSUAL();
        ldy = N;
    } else {
        if (!look(out, dtype, device, &t) || !rows_of(&t, M, N, &ldy)) UNUSUAL();
        y = t.data;
        Py_INCREF(out);
    }
    if (!scratch(need, a[0], &hold, &ws)) {
        Py_DECREF(out);
        UNUSUAL();
    }
    int st;
    LAUNCH(st, grouped ? lib.expert_linear_forward(kind, (int)M, (int)N, (int)K, (int)E, offsets, x.data, ldx, w.data, m.ld,
                                                   m.expert, m.order, bias, residual, ldr, act, z, ldz, y, ldy, ws, need, stream)
                       : lib.linear_forward(kind, (int)M, (int)N, (int)K, x.data, ldx, w.data, m.ld, m.order, bias, residual,
                                            ldr, act, z, ldz, y, ldy, ws, need, stream));
    Py_XDECREF(hold);
    if (st == 0) return out;
    Py_DECREF(out);
    return PyLong_FromLong(st);
}

/* backward(dy, x, w, offsets, preact, activation, need_dx, need_dw, need_dbias) -> (dx, dw, dbias) */
static PyObject *backward(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    PyObject *dtype, *dx = NULL, *dw = NULL, *db = NULL, *hold = NULL, *result = NULL;
    int64_t device, lddy, ldx, ldz = 0;
    stream_t stream;
    int act;
    Tensor g, x, w, t;
    Weight m;
    const void *z = NULL;
    void *dxp = NULL, *dwp = NULL, *dbp = NULL, *ws = NULL;
    if (n != 9) UNUSUAL();
    const int kind = kind_of(a[1], &dtype);
    if (kind < 0 || !here(a[1], &device, &stream) || !look(a[0], dtype, device, &g) || !look(a[1], dtype, device, &x) ||
        !look(a[2], dtype, device, &w) || !activation(a[5], &act) || (a[4] == Py_None) != (act == 0))
        UNUSUAL();
    const int grouped = a[3] != Py_None;
    if (x.dims != 2 || !weight_of(&w, 2 + grouped, &m)) UNUSUAL();
    const int64_t M = x.size[0], K = m.K, N = m.N, E = grouped ? w.size[0] : 0;
    if (!small(M, N, K) || E > INT32_MAX || !rows_of(&x, M, K, &ldx) || !rows_of(&g, M, N, &lddy)) UNUSUAL();
    const int *offsets = NULL;
    if (grouped) {
        if (!look(a[3], int32_type, device, &t) || !flat(&t, 1, E + 1, 0)) UNUSUAL();
        offsets = t.data;
    }
    if (a[4] != Py_None) {
        if (!look(a[4], dtype, device, &t) || !rows_of(&t, M, N, &ldz)) UNUSUAL();
        z = t.data;
    }
    const int want_dx = a[6] == Py_True, want_dw = a[7] == Py_True, want_db = a[8] == Py_True;
    if ((!want_dx && a[6] != Py_False) || (!want_dw && a[7] != Py_False) || (!want_db && a[8] != Py_False)) UNUSUAL();
    const size_t need =
        grouped ? lib.expert_linear_backward_workspace_size(kind, (int)M, (int)N, (int)K, (int)E, g.data, lddy, x.data, ldx,
                                                            w.data, m.ld, m.expert, m.order, act, want_dx, want_dw, want_db)
                : lib.linear_backward_workspace_size(kind, (int)M, (int)N, (int)K, g.data, lddy, x.data, ldx, w.data, m.ld,
                                                     m.order, act, want_dx, want_dw, want_db);
    const int64_t dx_size[2] = {M, K}, dw_size[3] = {E, m.order ? N : K, m.order ? K : N}, db_size[2] = {E, N};
    if (want_dx && (dx = new_tensor(2, dx_size, dtype, a[1], &dxp)) == NULL) goto unusual;
    if (want_dw && (dw = new_tensor(2 + grouped, dw_size + !grouped, dtype, a[1], &dwp)) == NULL) goto unusual;
    if (want_db && (db = new_tensor(1 + grouped, db_size + !grouped, dtype, a[1], &dbp)) == NULL) goto unusual;
    if (want_dw && m.order) {
        PyObject *args[3] = {dw, minus1, minus2};
        PyObject *turned = PyObject_VectorcallMethod(s_transpose, args, 3 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
        Py_DECREF(dw);
        dw = turned;
        if (dw == NULL) goto unusual;
    }
    if (!scratch(need, a[1], &hold, &ws)) goto unusual;
    const int64_t lddw = m.order ? K : N;
    int st;
    LAUNCH(st, grouped ? lib.expert_linear_backward(kind, (int)M, (int)N, (int)K, (int)E, offsets, g.data, lddy, x.data, ldx,
                                                    w.data, m.ld, m.expert, m.order, z, ldz, act, dxp, K, dwp, lddw, K * N,
                                                    dbp, ws, need, stream)
                       : lib.linear_backward(kind, (int)M, (int)N, (int)K, g.data, lddy, x.data, ldx, w.data, m.ld, m.order, z,
                                             ldz, act, dxp, K, dwp, lddw, dbp, ws, need, stream));
    Py_XDECREF(hold);
    if (st == 0)
        result = PyTuple_Pack(3, dx != NULL ? dx : Py_None, dw != NULL ? dw : Py_None, db != NULL ? db : Py_None);
    else
        result = PyLong_FromLong(st);
    Py_XDECREF(dx);
    Py_XDECREF(dw);
    Py_XDECREF(db);
    return result;
unusual:
    Py_XDECREF(dx);
    Py_XDECREF(dw);
    Py_XDECREF(db);
    UNUSUAL();
}

/* sort(choices, experts) -> (rows, offsets) */
static PyObject *sort(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    int64_t device, E;
    stream_t stream;
    Tensor c;
    void *rp, *op, *ws;
    if (n != 2 || !PyObject_TypeCheck(a[0], (PyTypeObject *)tensor_type) || !PyLong_CheckExact(a[1]) || !whole(a[1], &E) ||
        E < 1 || E > INT32_MAX - 1)
        UNUSUAL();
    PyObject *d = PyObject_GetAttr(a[0], s_dtype);
    Py_XDECREF(d);
    if ((d != int32_type && d != int64_type) || !here(a[0], &device, &stream) || !look(a[0], d, device, &c) || c.dims != 2 ||
        !flat(&c, 2, c.size[0], c.size[1]) || !small(c.size[0], c.size[1], 0))
        UNUSUAL();
    const int T = (int)c.size[0], J = (int)c.size[1];
    const size_t need = lib.expert_sort_workspace_size(T, J, (int)E);
    const int64_t o_size[1] = {E + 1};
    PyObject *rows = new_tensor(2, c.size, int32_type, a[0], &rp);
    PyObject *offsets = rows == NULL ? NULL : new_tensor(1, o_size, int32_type, a[0], &op);
    PyObject *hold = NULL;
    if (offsets == NULL || !scratch(need, a[0], &hold, &ws)) {
        Py_XDECREF(rows);
        Py_XDECREF(offsets);
        UNUSUAL();
    }
    int st;
    LAUNCH(st, lib.expert_sort(T, J, (int)E, c.data, d == int32_type ? 4 : 8, rp, op, ws, need, stream));
    Py_XDECREF(hold);
    PyObject *result = st == 0 ? PyTuple_Pack(2, rows, offsets) : PyLong_FromLong(st);
    Py_DECREF(rows);
    Py_DECREF(offsets);
    return result;
}

/* rows (T, J) and offsets (E + 1,) of a route. */
static int order_of(PyObject *rows, PyObject *offsets, int64_t device, int64_t *T, int64_t *J, int64_t *E, const int **r,
                    const int **o) {
    Tensor t;
    if (!look(rows, int32_type, device, &t) || t.dims != 2 || !flat(&t, 2, t.size[0], t.size[1]) ||
        !small(t.size[0], t.size[1], 0))
        return 0;
    *T = t.size[0];
    *J = t.size[1];
    *r = t.data;
    if (offsets == NULL) return 1;
    if (!look(offsets, int32_type, device, &t) || t.dims != 1 || !flat(&t, 1, t.size[0], 0) || !small(t.size[0], 0, 0)) return 0;
    *E = t.size[0] - 1;
    *o = t.data;
    return 1;
}

/* gather(x, rows, offsets, out) -> out */
static PyObject *gather(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    PyObject *dtype;
    int64_t device, T, J, E, ldx, lds;
    stream_t stream;
    Tensor x, t;
    const int *rows, *offsets;
    void *xs;
    if (n != 4) UNUSUAL();
    const int kind = kind_of(a[0], &dtype);
    if (kind < 0 || !here(a[0], &device, &stream) || !look(a[0], dtype, device, &x) || x.dims != 2 ||
        !order_of(a[1], a[2], device, &T, &J, &E, &rows, &offsets) || E < 0 || !rows_of(&x, T, x.size[1], &ldx) ||
        !small(x.size[1], 0, 0))
        UNUSUAL();
    const int64_t H = x.size[1], size[2] = {T * J, H};
    PyObject *out = a[3];
    if (out == Py_None) {
        out = new_tensor(2, size, dtype, a[0], &xs);
        if (out == NULL) UNUSUAL();
        lds = H > 1 ? H : 1;
    } else {
        if (!look(out, dtype, device, &t) || !rows_of(&t, T * J, H, &lds)) UNUSUAL();
        xs = t.data;
        Py_INCREF(out);
    }
    int st;
    LAUNCH(st, lib.expert_gather(kind, (int)T, (int)J, (int)H, (int)E, rows, offsets, x.data, ldx, xs, lds, stream));
    if (st == 0) return out;
    Py_DECREF(out);
    return PyLong_FromLong(st);
}

static int weights_of(PyObject *o, int64_t device, int64_t T, int64_t J, const float **w) {
    Tensor t;
    *w = NULL;
    if (o == Py_None) return 1;
    if (!look(o, kinds[0], device, &t) || !flat(&t, 2, T, J)) return 0;
    *w = t.data;
    return 1;
}

/* combine(ys, rows, weights, residual, out) -> out */
static PyObject *combine(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    PyObject *dtype;
    int64_t device, T, J, E, lds, ldr = 0, ldy;
    stream_t stream;
    Tensor s, t;
    const int *rows, *none;
    const float *weights;
    const void *residual = NULL;
    void *y;
    if (n != 5) UNUSUAL();
    const int kind = kind_of(a[0], &dtype);
    if (kind < 0 || !here(a[0], &device, &stream) || !look(a[0], dtype, device, &s) || s.dims != 2 ||
        !order_of(a[1], NULL, device, &T, &J, &E, &rows, &none) || !rows_of(&s, T * J, s.size[1], &lds) ||
        !small(s.size[1], 0, 0) || !weights_of(a[2], device, T, J, &weights))
        UNUSUAL();
    const int64_t H = s.size[1], size[2] = {T, H};
    if (a[3] != Py_None) {
        if (!look(a[3], dtype, device, &t) || !rows_of(&t, T, H, &ldr)) UNUSUAL();
        residual = t.data;
    }
    PyObject *out = a[4];
    if (out == Py_None) {
        out = new_tensor(2, size, dtype, a[0], &y);
        if (out == NULL) UNUSUAL();
        ldy = H > 1 ? H : 1;
    } else {
        if (!look(out, dtype, device, &t) || !rows_of(&t, T, H, &ldy)) UNUSUAL();
        y = t.data;
        Py_INCREF(out);
    }
    int st;
    LAUNCH(st, lib.expert_combine(kind, (int)T, (int)J, (int)H, rows, weights, s.data, lds, residual, ldr, y, ldy, stream));
    if (st == 0) return out;
    Py_DECREF(out);
    return PyLong_FromLong(st);
}

/* combine_backward(dy, ys, rows, weights, offsets, need_dweights) -> (dys, dweights) */
static PyObject *combine_backward(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    PyObject *dtype, *dw = NULL;
    int64_t device, T, J, E, lddy, lds = 0;
    stream_t stream;
    Tensor g, t;
    const int *rows, *offsets;
    const float *weights;
    const void *ys = NULL;
    void *dysp, *dwp = NULL;
    if (n != 6) UNUSUAL();
    const int kind = kind_of(a[0], &dtype), want = a[5] == Py_True;
    if (kind < 0 || (!want && a[5] != Py_False) || !here(a[0], &device, &stream) || !look(a[0], dtype, device, &g) ||
        g.dims != 2 || !order_of(a[2], a[4], device, &T, &J, &E, &rows, &offsets) || E < 0 ||
        !rows_of(&g, T, g.size[1], &lddy) || !small(g.size[1], 0, 0) || !weights_of(a[3], device, T, J, &weights))
        UNUSUAL();
    const int64_t H = g.size[1], size[2] = {T * J, H}, w_size[2] = {T, J};
    if (want) {
        if (!look(a[1], dtype, device, &t) || !rows_of(&t, T * J, H, &lds)) UNUSUAL();
        ys = t.data;
    }
    PyObject *dys = new_tensor(2, size, dtype, a[0], &dysp);
    if (dys != NULL && want) dw = new_tensor(2, w_size, kinds[0], a[0], &dwp);
    if (dys == NULL || (want && dw == NULL)) {
        Py_XDECREF(dys);
        UNUSUAL();
    }
    int st;
    LAUNCH(st, lib.expert_combine_backward(kind, (int)T, (int)J, (int)H, (int)E, rows, offsets, weights, g.data, lddy, ys, lds,
                                           dysp, H > 1 ? H : 1, dwp, stream));
    PyObject *result = st == 0 ? PyTuple_Pack(2, dys, dw != NULL ? dw : Py_None) : PyLong_FromLong(st);
    Py_DECREF(dys);
    Py_XDECREF(dw);
    return result;
}

/* float32 (M,), or NULL for None; 0 for anything else */
static int floats_of(PyObject *o, int64_t device, int64_t M, const float **p) {
    Tensor t;
    *p = NULL;
    if (o == Py_None) return 1;
    if (!look(o, kinds[0], device, &t) || !flat(&t, 1, M, 0)) return 0;
    *p = t.data;
    return 1;
}
/* A vector (N,) of this type, or NULL for None. */
static int vector_of(PyObject *o, PyObject *dtype, int64_t device, int64_t N, const void **p) {
    Tensor t;
    *p = NULL;
    if (o == Py_None) return 1;
    if (!look(o, dtype, device, &t) || !flat(&t, 1, N, 0)) return 0;
    *p = t.data;
    return 1;
}
static int truth(PyObject *o, int *v) {
    *v = o == Py_True;
    return *v || o == Py_False;
}
static int scoring_of(PyObject *name, int *v) {
    int64_t n;
    if (!whole(PyDict_GetItemWithError(scorings, name), &n)) return 0;
    *v = (int)n;
    return 1;
}
static int small_number(PyObject *o, int *v) {
    int64_t n;
    if (!PyLong_CheckExact(o) || !whole(o, &n) || n < INT32_MIN || n > INT32_MAX) return 0;
    *v = (int)n;
    return 1;
}

/* norm(x, weight, bias, eps, stats, out) -> out */
static PyObject *norm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    PyObject *dtype;
    int64_t device, ldx, ldy;
    stream_t stream;
    Tensor x, t;
    const void *weight, *bias;
    float *stats = NULL;
    void *y;
    if (n != 6 || scorings == NULL || !PyFloat_CheckExact(a[3])) UNUSUAL();
    const int kind = kind_of(a[0], &dtype);
    if (kind < 0 || !here(a[0], &device, &stream) || !look(a[0], dtype, device, &x) || x.dims != 2 ||
        !rows_of(&x, x.size[0], x.size[1], &ldx) || !small(x.size[0], x.size[1], 0))
        UNUSUAL();
    const int64_t M = x.size[0], N = x.size[1];
    if (!vector_of(a[1], dtype, device, N, &weight) || !vector_of(a[2], dtype, device, N, &bias)) UNUSUAL();
    if (a[4] != Py_None) {
        if (!look(a[4], kinds[0], device, &t) || !flat(&t, 2, M, 2)) UNUSUAL();
        stats = t.data;
    }
    PyObject *out = a[5];
    if (out == Py_None) {
        out = new_tensor(2, x.size, dtype, a[0], &y);
        if (out == NULL) UNUSUAL();
        ldy = N > 1 ? N : 1;
    } else {
        if (!look(out, dtype, device, &t) || !rows_of(&t, M, N, &ldy)) UNUSUAL();
        y = t.data;
        Py_INCREF(out);
    }
    int st;
    LAUNCH(st, more.layer_norm_forward(kind, (int)M, (int)N, x.data, ldx, weight, bias, (float)PyFloat_AS_DOUBLE(a[3]), stats, y, ldy,
                                       stream));
    if (st == 0) return out;
    Py_DECREF(out);
    return PyLong_FromLong(st);
}

/* norm_backward(dy, x, weight, stats, need_dx, need_dweight, need_dbias) -> (dx, dweight, dbias) */
static PyObject *norm_backward(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    PyObject *dtype, *made[3] = {NULL, NULL, NULL}, *hold = NULL, *result = NULL;
    int64_t device, lddy, ldx;
    stream_t stream;
    Tensor g, x, t;
    const void *weight;
    void *p[3] = {NULL, NULL, NULL}, *ws = NULL;
    int want[3];
    if (n != 7 || scorings == NULL) UNUSUAL();
    const int kind = kind_of(a[1], &dtype);
    if (kind < 0 || !here(a[1], &device, &stream) || !look(a[1], dtype, device, &x) || !look(a[0], dtype, device, &g) || x.dims != 2)
        UNUSUAL();
    const int64_t M = x.size[0], N = x.size[1];
    if (!small(M, N, 0) || !rows_of(&x, M, N, &ldx) || !rows_of(&g, M, N, &lddy) || !vector_of(a[2], dtype, device, N, &weight) ||
        !look(a[3], kinds[0], device, &t) || !flat(&t, 2, M, 2) || !truth(a[4], &want[0]) || !truth(a[5], &want[1]) ||
        !truth(a[6], &want[2]))
        UNUSUAL();
    const size_t need = more.layer_norm_backward_workspace_size((int)M, (int)N, want[1], want[2]);
    int ok = 1;
    for (int i = 0; i < 3 && ok; ++i)
        if (want[i]) ok = (made[i] = new_tensor(i == 0 ? 2 : 1, x.size + (i == 0 ? 0 : 1), dtype, a[1], &p[i])) != NULL;
    if (ok && scratch(need, a[1], &hold, &ws)) {
        int st;
        LAUNCH(st, more.layer_norm_backward(kind, (int)M, (int)N, g.data, lddy, x.data, ldx, weight, t.data, p[0], N > 1 ? N : 1, p[1],
                                            p[2], ws, need, stream));
        Py_XDECREF(hold);
        result = st != 0 ? PyLong_FromLong(st)
                         : PyTuple_Pack(3, want[0] ? made[0] : Py_None, want[1] ? made[1] : Py_None, want[2] ? made[2] : Py_None);
    }
    for (int i = 0; i < 3; ++i) Py_XDECREF(made[i]);
    if (result == NULL) UNUSUAL();
    return result;
}

/* choose(logits, choices, bias, scoring, groups, kept_groups, group_top, renormalize, scale) -> (chosen, weights) */
static PyObject *choose(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    PyObject *dtype;
    int64_t device, ld;
    stream_t stream;
    Tensor l;
    const float *bias;
    int J, how, groups, kept, top, renormalize;
    void *cp, *wp;
    if (n != 9 || scorings == NULL || !PyFloat_CheckExact(a[8])) UNUSUAL();
    const int kind = kind_of(a[0], &dtype);
    if (kind < 0 || !here(a[0], &device, &stream) || !look(a[0], dtype, device, &l) || l.dims != 2 ||
        !rows_of(&l, l.size[0], l.size[1], &ld) || !small(l.size[0], l.size[1], 0) || !floats_of(a[2], device, l.size[1], &bias) ||
        !small_number(a[1], &J) || J < 0 || !scoring_of(a[3], &how) || !small_number(a[4], &groups) || !small_number(a[5], &kept) ||
        !small_number(a[6], &top) || !truth(a[7], &renormalize))
        UNUSUAL();
    const int64_t size[2] = {l.size[0], J};
    PyObject *chosen = new_tensor(2, size, int32_type, a[0], &cp);
    PyObject *weights = chosen == NULL ? NULL : new_tensor(2, size, kinds[0], a[0], &wp);
    if (weights == NULL) {
        Py_XDECREF(chosen);
        UNUSUAL();
    }
    int st;
    LAUNCH(st, more.expert_choose(kind, (int)l.size[0], (int)l.size[1], J, l.data, ld, bias, how, groups, kept, top, renormalize,
                                  (float)PyFloat_AS_DOUBLE(a[8]), cp, wp, stream));
    PyObject *result = st == 0 ? PyTuple_Pack(2, chosen, weights) : PyLong_FromLong(st);
    Py_DECREF(chosen);
    Py_DECREF(weights);
    return result;
}

/* choose_backward(dweights, logits, chosen, scoring, renormalize, scale) -> dlogits */
static PyObject *choose_backward(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    PyObject *dtype;
    int64_t device, ld;
    stream_t stream;
    Tensor l, c, g;
    int how, renormalize;
    void *dp;
    if (n != 6 || scorings == NULL || !PyFloat_CheckExact(a[5])) UNUSUAL();
    const int kind = kind_of(a[1], &dtype);
    if (kind < 0 || !here(a[1], &device, &stream) || !look(a[1], dtype, device, &l) || l.dims != 2 ||
        !rows_of(&l, l.size[0], l.size[1], &ld) || !small(l.size[0], l.size[1], 0) || !look(a[2], int32_type, device, &c) ||
        c.dims != 2 || !flat(&c, 2, l.size[0], c.size[1]) || !small(c.size[1], 0, 0) || !look(a[0], kinds[0], device, &g) ||
        !flat(&g, 2, l.size[0], c.size[1]) || !scoring_of(a[3], &how) || !truth(a[4], &renormalize))
        UNUSUAL();
    PyObject *d = new_tensor(2, l.size, dtype, a[1], &dp);
    if (d == NULL) UNUSUAL();
    int st;
    LAUNCH(st, more.expert_choose_backward(kind, (int)l.size[0], (int)l.size[1], (int)c.size[1], g.data, c.data, l.data, ld, how,
                                           renormalize, (float)PyFloat_AS_DOUBLE(a[5]), dp, l.size[1] > 1 ? l.size[1] : 1, stream));
    if (st == 0) return d;
    Py_DECREF(d);
    return PyLong_FromLong(st);
}

/* What both calls of a head's loss take: x, w and targets. */
typedef struct {
    PyObject *dtype;
    int64_t device, M, N, K, ldx;
    stream_t stream;
    Tensor x, w, t;
    Weight m;
    int kind, target_bytes;
} Head;
static int head_of(PyObject *x, PyObject *w, PyObject *targets, Head *h) {
    h->kind = kind_of(x, &h->dtype);
    if (h->kind < 0 || !here(x, &h->device, &h->stream) || !look(x, h->dtype, h->device, &h->x) ||
        !look(w, h->dtype, h->device, &h->w) || h->x.dims != 2 || !weight_of(&h->w, 2, &h->m) ||
        !rows_of(&h->x, h->x.size[0], h->m.K, &h->ldx) || !PyObject_TypeCheck(targets, (PyTypeObject *)tensor_type))
        return 0;
    h->M = h->x.size[0], h->K = h->m.K, h->N = h->m.N;
    PyObject *d = PyObject_GetAttr(targets, s_dtype);
    Py_XDECREF(d);
    h->target_bytes = d == int32_type ? 4 : 8;
    return (d == int32_type || d == int64_type) && look(targets, d, h->device, &h->t) && flat(&h->t, 1, h->M, 0) &&
           small(h->M, h->N, h->K);
}

/* cross_entropy(x, w, targets) -> (loss, lse) */
static PyObject *cross_entropy(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Head h;
    void *lp, *ep, *ws;
    PyObject *hold = NULL;
    if (n != 3 || scorings == NULL || !head_of(a[0], a[1], a[2], &h)) UNUSUAL();
    const size_t need = more.linear_cross_entropy_forward_workspace_size(h.kind, (int)h.M, (int)h.N, (int)h.K, h.x.data, h.ldx, h.w.data,
                                                                         h.m.ld, h.m.order);
    PyObject *loss = new_tensor(1, &h.M, kinds[0], a[0], &lp);
    PyObject *lse = loss == NULL ? NULL : new_tensor(1, &h.M, kinds[0], a[0], &ep);
    if (lse == NULL || !scratch(need, a[0], &hold, &ws)) {
        Py_XDECREF(loss);
        Py_XDECREF(lse);
        UNUSUAL();
    }
    int st;
    LAUNCH(st, more.linear_cross_entropy_forward(h.kind, (int)h.M, (int)h.N, (int)h.K, h.x.data, h.ldx, h.w.data, h.m.ld, h.m.order,
                                                 h.t.data, h.target_bytes, lp, ep, ws, need, h.stream));
    Py_XDECREF(hold);
    PyObject *result = st == 0 ? PyTuple_Pack(2, loss, lse) : PyLong_FromLong(st);
    Py_DECREF(loss);
    Py_DECREF(lse);
    return result;
}

/* cross_entropy_backward(dloss, x, w, targets, lse, dlse, need_dx, need_dw) -> (dx, dw) */
static PyObject *cross_entropy_backward(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    Head h;
    const float *dloss, *dlse, *lse;
    int want_dx, want_dw;
    void *dxp = NULL, *dwp = NULL, *ws = NULL;
    PyObject *dx = NULL, *dw = NULL, *hold = NULL, *result = NULL;
    if (n != 8 || scorings == NULL || a[4] == Py_None || !head_of(a[1], a[2], a[3], &h) || !floats_of(a[0], h.device, h.M, &dloss) ||
        !floats_of(a[4], h.device, h.M, &lse) || !floats_of(a[5], h.device, h.M, &dlse) || !truth(a[6], &want_dx) ||
        !truth(a[7], &want_dw))
        UNUSUAL();
    const size_t need = more.linear_cross_entropy_backward_workspace_size(h.kind, (int)h.M, (int)h.N, (int)h.K, h.x.data, h.ldx,
                                                                          h.w.data, h.m.ld, h.m.order, want_dx, want_dw);
    const int64_t dx_size[2] = {h.M, h.K}, dw_size[2] = {h.m.order ? h.N : h.K, h.m.order ? h.K : h.N};
    int ok = !want_dx || (dx = new_tensor(2, dx_size, h.dtype, a[1], &dxp)) != NULL;
    ok = ok && (!want_dw || (dw = new_tensor(2, dw_size, h.dtype, a[1], &dwp)) != NULL);
    if (ok && want_dw && h.m.order) {
        PyObject *args[3] = {dw, minus1, minus2};
        PyObject *turned = PyObject_VectorcallMethod(s_transpose, args, 3 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
        Py_DECREF(dw);
        dw = turned;
        ok = dw != NULL;
    }
    if (ok && scratch(need, a[1], &hold, &ws)) {
        int st;
        LAUNCH(st, more.linear_cross_entropy_backward(h.kind, (int)h.M, (int)h.N, (int)h.K, dloss, dlse, h.x.data, h.ldx, h.w.data,
                                                      h.m.ld, h.m.order, h.t.data, h.target_bytes, lse, dxp, h.K, dwp, dw_size[1], ws,
                                                      need, h.stream));
        Py_XDECREF(hold);
        result = st == 0 ? PyTuple_Pack(2, want_dx ? dx : Py_None, want_dw ? dw : Py_None) : PyLong_FromLong(st);
    }
    Py_XDECREF(dx);
    Py_XDECREF(dw);
    if (result == NULL) UNUSUAL();
    return result;
}

static int addresses(PyObject *functions, const char *const *names, size_t n, void **slots) {
    for (size_t i = 0; i < n; ++i) {
        PyObject *v = PyDict_GetItemString(functions, names[i]);
        if (v == NULL) {
            PyErr_Format(PyExc_KeyError, "%s", names[i]);
            return 0;
        }
        slots[i] = PyLong_AsVoidPtr(v);
        if (slots[i] == NULL) {
            if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s", names[i]);
            return 0;
        }
    }
    return 1;
}

/* bind_more(functions: dict of addresses, scorings: dict), after bind(); without it
 * the operators around the layers answer NotImplemented */
static PyObject *bind_more(PyObject *self, PyObject *args) {
    PyObject *functions, *names;
    _Static_assert(sizeof more == sizeof more_names / sizeof *more_names * sizeof(void *), "a name for each function");
    if (!PyArg_ParseTuple(args, "O!O!", &PyDict_Type, &functions, &PyDict_Type, &names) ||
        !addresses(functions, more_names, sizeof more_names / sizeof *more_names, (void **)&more))
        return NULL;
    scorings = Py_NewRef(names);
    Py_RETURN_NONE;
}

/* bind(functions: dict of addresses, objects: tuple) */
static PyObject *bind(PyObject *self, PyObject *args) {
    PyObject *functions, *objects;
    _Static_assert(sizeof lib == sizeof lib_names / sizeof *lib_names * sizeof(void *), "a name for each function");
    if (!PyArg_ParseTuple(args, "O!O!", &PyDict_Type, &functions, &PyTuple_Type, &objects) ||
        !addresses(functions, lib_names, sizeof lib_names / sizeof *lib_names, (void **)&lib))
        return NULL;
    if (!PyArg_ParseTuple(objects, "OOOOO!(OOO)OOO", &tensor_type, &empty, &raw_stream, &get_device, &PyDict_Type, &activations,
                          &kinds[0], &kinds[1], &kinds[2], &int32_type, &int64_type, &uint8_type))
        return NULL;
    if (!PyType_Check(tensor_type)) return PyErr_Format(PyExc_TypeError, "the tensor type is none");
    Py_INCREF(objects); /* and with it all of them, for good */
    s_dtype = PyUnicode_InternFromString("dtype");
    s_device = PyUnicode_InternFromString("device");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_transpose = PyUnicode_InternFromString("transpose");
    empty_names = Py_BuildValue("(ss)", "dtype", "device");
    minus1 = PyLong_FromLong(-1);
    minus2 = PyLong_FromLong(-2);
    if (PyErr_Occurred()) return NULL;
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, NULL},
                                {"bind_more", bind_more, METH_VARARGS, NULL},
                                {"norm", (PyCFunction)(void (*)(void))norm, METH_FASTCALL, NULL},
                                {"norm_backward", (PyCFunction)(void (*)(void))norm_backward, METH_FASTCALL, NULL},
                                {"choose", (PyCFunction)(void (*)(void))choose, METH_FASTCALL, NULL},
                                {"choose_backward", (PyCFunction)(void (*)(void))choose_backward, METH_FASTCALL, NULL},
                                {"cross_entropy", (PyCFunction)(void (*)(void))cross_entropy, METH_FASTCALL, NULL},
                                {"cross_entropy_backward", (PyCFunction)(void (*)(void))cross_entropy_backward, METH_FASTCALL, NULL},
                                {"forward", (PyCFunction)(void (*)(void))forward, METH_FASTCALL, NULL},
                                {"backward", (PyCFunction)(void (*)(void))backward, METH_FASTCALL, NULL},
                                {"sort", (PyCFunction)(void (*)(void))sort, METH_FASTCALL, NULL},
                                {"gather", (PyCFunction)(void (*)(void))gather, METH_FASTCALL, NULL},
                                {"combine", (PyCFunction)(void (*)(void))combine, METH_FASTCALL, NULL},
                                {"combine_backward", (PyCFunction)(void (*)(void))combine_backward, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast_call", NULL, -1, methods};
PyMODINIT_FUNC PyInit__fast_call(void) { return PyModule_Create(&module); }
