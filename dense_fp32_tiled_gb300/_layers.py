"""Layer operators on torch tensors: argument marshalling for include/linear.h
and include/experts.h.  As in ``_binding``, every arithmetic step runs in the
CUDA library; PyTorch supplies device memory, strides and the current stream.

Every function runs on ``stream`` (a torch.cuda.Stream) or the current one, is
asynchronous, and allocates what it returns on that stream.  Tensors of one
call share a device and a type (float32, bfloat16 or float16).  Wrong shapes
and types raise ValueError and TypeError before anything is launched; a
status of the library raises SgemmError.
"""
from __future__ import annotations

import contextlib

from ._binding import SGEMM_OK, SgemmError, _workspace, load_library

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
_types = {}


def _type_of(t, name):
    import torch
    if not _types:
        _types.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in _types:
        raise TypeError(f"{name} must be a CUDA tensor of float32, bfloat16 or float16")
    return _types[t.dtype]


def _like(t, ref, name):
    if getattr(t, "dtype", None) != ref.dtype or t.device != ref.device:
        raise TypeError(f"{name} must be a {ref.dtype} tensor on {ref.device}")


def _rows(t, rows, cols, name, ref=None):
    """(address, row stride) of a row-major rows x cols tensor."""
    if ref is not None:
        _like(t, ref, name)
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError(f"{name} must have shape ({rows}, {cols}), got {tuple(t.shape)}")
    ld, inner = t.stride()
    if cols > 1 and inner != 1:
        raise ValueError(f"{name} must be row-major with unit column stride")
    if rows <= 1:
        ld = max(ld, cols, 1)
    elif ld < cols:
        raise ValueError(f"{name} has overlapping rows")
    return t.data_ptr(), max(ld, 1)


def _vector(t, shape, name, ref):
    if t is None:
        return None
    _like(t, ref, name)
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {shape}, got {tuple(t.shape)}")
    return t.data_ptr()


def _weight(w, K, N, name, ref=None):
    """(address, stride, order, expert stride) of (..., K, N) with either of the last two contiguous."""
    if ref is not None:
        _like(w, ref, name)
    if w.shape[-2] != K or w.shape[-1] != N:
        raise ValueError(f"{name} must end in ({K}, {N}), got {tuple(w.shape)}")
    sk, sn = w.stride()[-2:]
    expert = w.stride(0) if w.dim() == 3 and w.shape[0] > 1 else 0
    if (sn == 1 or N == 1) and (K <= 1 or sk >= N):
        return w.data_ptr(), (max(sk, N, 1) if K <= 1 else sk), 0, expert
    if (sk == 1 or K == 1) and (N <= 1 or sn >= K):
        return w.data_ptr(), (max(sn, K, 1) if N <= 1 else sn), 1, expert
    raise ValueError(f"{name} must have one of its last two dimensions contiguous, its rows apart")


def _int32(t, shape, name, ref):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != ref.device:
        raise TypeError(f"{name} must be an int32 tensor on {ref.device}")
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {shape}, got {tuple(t.shape)}")
    return t.data_ptr()


class _On:
    """The device and stream of a call; what is allocated inside belongs to that stream."""

    __slots__ = ("stream", "_stack")

    def __init__(self, device, stream):
        import torch
        self._stack = None
        here = torch.cuda.current_device() == device.index
        if stream is None:
            self.stream = torch.cuda.current_stream(device)
            if not here:
                self._stack = contextlib.ExitStack()
                self._stack.enter_context(torch.cuda.device(device))
        else:
            self.stream = stream
            self._stack = contextlib.ExitStack()
            self._stack.enter_context(torch.cuda.stream(stream))

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        if self._stack is not None:
            self._stack.__exit__(*exc)
        return False

    def workspace(self, device, nbytes):
        return _workspace("layer", device, self.stream, nbytes).data_ptr() if nbytes else None


def _act(name):
    try:
        return ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {name!r}") from None


def _check(st, what):
    if st != SGEMM_OK:
        raise SgemmError(st, what)


# ---- the product with its epilogue ---------------------------------------------
def linear(x, w, bias=None, residual=None, activation="none", preact=None, out=None, stream=None):
    """act(x @ w + bias) + residual.

    x is (M, K), row-major with any row stride; w is (K, N) in either memory
    order (``weight.t()`` of an (N, K) weight is read as it is); bias is (N,);
    residual and out are (M, N).  ``preact``, an (M, N) tensor, receives
    x @ w + bias for linear_backward.  ``out`` may be ``residual`` itself.
    """
    return _forward(x, w, None, bias, residual, activation, preact, out, stream)


def expert_linear(x, w, offsets, bias=None, residual=None, activation="none", preact=None, out=None, stream=None):
    """The same product over rows sorted by expert: rows offsets[e] to
    offsets[e + 1] of x (R, K) meet w[e] and bias[e] of w (E, K, N) and bias
    (E, N).  offsets is int32 (E + 1,) on the device, as expert_sort makes it,
    and is not read on the host.  Rows of no expert give 0."""
    return _forward(x, w, offsets, bias, residual, activation, preact, out, stream)


def _forward(x, w, offsets, bias, residual, activation, preact, out, stream):
    import torch
    kind, act = _type_of(x, "x"), _act(activation)
    grouped = offsets is not None
    if x.dim() != 2 or w.dim() != 2 + grouped:
        raise ValueError(f"x must be 2-D and w {2 + grouped}-D, got {tuple(x.shape)} and {tuple(w.shape)}")
    M, K = x.shape
    N = w.shape[-1]
    xp, ldx = _rows(x, M, K, "x")
    wp, ldw, order, step = _weight(w, K, N, "w", x)
    rp, ldr = _rows(residual, M, N, "residual", x) if residual is not None else (None, 0)
    zp, ldz = _rows(preact, M, N, "preact", x) if preact is not None else (None, 0)
    lib = load_library()
    with _On(x.device, stream) as on:
        if out is None:
            out = torch.empty((M, N), dtype=x.dtype, device=x.device)
        yp, ldy = _rows(out, M, N, "out", x)
        if grouped:
            E = w.shape[0]
            op = _int32(offsets, (E + 1,), "offsets", x)
            bp = _vector(bias, (E, N), "bias", x)
            nbytes = lib.expert_linear_forward_workspace_size(kind, M, N, K, E, xp, ldx, wp, ldw, step, order)
            _check(lib.expert_linear_forward(kind, M, N, K, E, op, xp, ldx, wp, ldw, step, order, bp, rp, ldr, act, zp,
                                             ldz, yp, ldy, on.workspace(x.device, nbytes), nbytes,
                                             on.stream.cuda_stream), "expert_linear_forward")
        else:
            bp = _vector(bias, (N,), "bias", x)
            nbytes = lib.linear_forward_workspace_size(kind, M, N, K, xp, ldx, wp, ldw, order)
            _check(lib.linear_forward(kind, M, N, K, xp, ldx, wp, ldw, order, bp, rp, ldr, act, zp, ldz, yp, ldy,
                                      on.workspace(x.device, nbytes), nbytes, on.stream.cuda_stream),
                   "linear_forward")
    return out


def linear_backward(dy, x, w, preact=None, activation="none", need_dx=True, need_dw=True, need_dbias=True, stream=None):
    """(dx, dw, dbias) of linear for the gradient dy of its result (that of the
    residual is dy itself).  preact is what linear saved, needed unless the
    activation is "none".  dw has the memory order of w; what is not needed is None."""
    return _backward(dy, x, w, None, preact, activation, need_dx, need_dw, need_dbias, stream)


def expert_linear_backward(dy, x, w, offsets, preact=None, activation="none", need_dx=True, need_dw=True,
                           need_dbias=True, stream=None):
    """(dx, dw, dbias) of expert_linear.  Rows of no expert have a dx of 0, experts without rows a dw and dbias of 0."""
    return _backward(dy, x, w, offsets, preact, activation, need_dx, need_dw, need_dbias, stream)


def _backward(dy, x, w, offsets, preact, activation, need_dx, need_dw, need_dbias, stream):
    import torch
    kind, act = _type_of(x, "x"), _act(activation)
    grouped = offsets is not None
    if x.dim() != 2 or w.dim() != 2 + grouped:
        raise ValueError(f"x must be 2-D and w {2 + grouped}-D, got {tuple(x.shape)} and {tuple(w.shape)}")
    if (preact is None) != (act == 0):
        raise ValueError("preact is needed with an activation, and only then")
    M, K = x.shape
    N = w.shape[-1]
    gp, lddy = _rows(dy, M, N, "dy", x)
    xp, ldx = _rows(x, M, K, "x")
    wp, ldw, order, step = _weight(w, K, N, "w", x)
    zp, ldz = _rows(preact, M, N, "preact", x) if preact is not None else (None, 0)
    lead = (w.shape[0],) if grouped else ()
    lib = load_library()
    with _On(x.device, stream) as on:
        dx = dw = dbias = None
        hp = ldh = vp = ldv = stepv = bp = None
        if need_dx:
            dx = torch.empty((M, K), dtype=x.dtype, device=x.device)
            hp = dx.data_ptr()
        if need_dw:
            if order == 0:
                dw = torch.empty(lead + (K, N), dtype=x.dtype, device=x.device)
            else:
                dw = torch.empty(lead + (N, K), dtype=x.dtype, device=x.device).transpose(-1, -2)
            vp = dw.data_ptr()
        if need_dbias:
            dbias = torch.empty(lead + (N,), dtype=x.dtype, device=x.device)
            bp = dbias.data_ptr()
        ldh, ldv, stepv = max(K, 1), max(K if order else N, 1), K * N
        if grouped:
            E = w.shape[0]
            op = _int32(offsets, (E + 1,), "offsets", x)
            nbytes = lib.expert_linear_backward_workspace_size(kind, M, N, K, E, gp, lddy, xp, ldx, wp, ldw, step, order,
                                                               act, need_dx, need_dw, need_dbias)
            _check(lib.expert_linear_backward(kind, M, N, K, E, op, gp, lddy, xp, ldx, wp, ldw, step, order, zp, ldz,
                                              act, hp, ldh, vp, ldv, stepv, bp, on.workspace(x.device, nbytes), nbytes,
                                              on.stream.cuda_stream), "expert_linear_backward")
        else:
            nbytes = lib.linear_backward_workspace_size(kind, M, N, K, gp, lddy, xp, ldx, wp, ldw, order, act, need_dx,
                                                        need_dw, need_dbias)
            _check(lib.linear_backward(kind, M, N, K, gp, lddy, xp, ldx, wp, ldw, order, zp, ldz, act, hp, ldh, vp, ldv,
                                       bp, on.workspace(x.device, nbytes), nbytes, on.stream.cuda_stream),
                   "linear_backward")
    return dx, dw, dbias


def linear_timeouts() -> int:
    """1 if a kernel of the layer products gave up a wait since the library was loaded, else 0."""
    import ctypes
    n = ctypes.c_uint()
    _check(load_library().linear_timeouts(ctypes.byref(n)), "linear_timeouts")
    return n.value


# ---- tokens to their experts and back --------------------------------------------
def expert_sort(choices, experts, stream=None):
    """(rows, offsets): choices is int32 or int64 (T, J), the experts of each
    token (one outside 0 .. experts - 1 is dropped).  rows, int32 (T, J), is
    each choice's place among all T*J sorted by expert, then token and choice,
    or -1; places offsets[e] to offsets[e + 1] belong to expert e."""
    import torch
    if not isinstance(choices, torch.Tensor) or not choices.is_cuda or choices.dtype not in (torch.int32, torch.int64):
        raise TypeError("choices must be a CUDA tensor of int32 or int64")
    if choices.dim() != 2 or not choices.is_contiguous():
        raise ValueError(f"choices must be contiguous with shape (tokens, choices), got {tuple(choices.shape)}")
    T, J = choices.shape
    E = int(experts)
    lib = load_library()
    with _On(choices.device, stream) as on:
        rows = torch.empty((T, J), dtype=torch.int32, device=choices.device)
        offsets = torch.empty((max(E, 0) + 1,), dtype=torch.int32, device=choices.device)
        nbytes = lib.expert_sort_workspace_size(T, J, E)
        _check(lib.expert_sort(T, J, E, choices.data_ptr(), choices.element_size(), rows.data_ptr(), offsets.data_ptr(),
                               on.workspace(choices.device, nbytes), nbytes, on.stream.cuda_stream), "expert_sort")
    return rows, offsets


def _order(rows, offsets, T, ref):
    if rows.dim() != 2 or rows.shape[0] != T:
        raise ValueError(f"rows must have shape ({T}, choices), got {tuple(rows.shape)}")
    if offsets is not None and offsets.dim() != 1:
        raise ValueError("offsets must be 1-D")
    J = rows.shape[1]
    E = offsets.shape[0] - 1 if offsets is not None else 0
    return J, E, _int32(rows, (T, J), "rows", ref), _int32(offsets, (E + 1,), "offsets", ref) if offsets is not None else None


def _weights(weights, T, J, ref):
    import torch
    if weights is None:
        return None
    if not isinstance(weights, torch.Tensor) or weights.dtype != torch.float32 or weights.device != ref.device:
        raise TypeError(f"weights must be a float32 tensor on {ref.device}")
    if tuple(weights.shape) != (T, J) or not weights.is_contiguous():
        raise ValueError(f"weights must be contiguous with shape ({T}, {J}), got {tuple(weights.shape)}")
    return weights.data_ptr()


def expert_gather(x, rows, offsets, out=None, stream=None):
    """The token rows in expert order: out[rows[t, j]] = x[t], (T*J, H); places in no use are 0."""
    import torch
    kind = _type_of(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got {tuple(x.shape)}")
    T, H = x.shape
    xp, ldx = _rows(x, T, H, "x")
    J, E, rp, op = _order(rows, offsets, T, x)
    with _On(x.device, stream) as on:
        if out is None:
            out = torch.empty((T * J, H), dtype=x.dtype, device=x.device)
        sp, lds = _rows(out, T * J, H, "out", x)
        _check(load_library().expert_gather(kind, T, J, H, E, rp, op, xp, ldx, sp, lds, on.stream.cuda_stream),
               "expert_gather")
    return out


def expert_combine(ys, rows, weights=None, residual=None, out=None, stream=None):
    """Each token's sum over its choices: residual[t] + sum_j weights[t, j] * ys[rows[t, j]].
    weights is float32 (T, J); None weighs all by 1.  Dropped choices add nothing."""
    import torch
    kind = _type_of(ys, "ys")
    if ys.dim() != 2 or rows.dim() != 2:
        raise ValueError(f"ys and rows must be 2-D, got {tuple(ys.shape)} and {tuple(rows.shape)}")
    T, H = rows.shape[0], ys.shape[1]
    J, _, rp, _ = _order(rows, None, T, ys)
    sp, lds = _rows(ys, T * J, H, "ys")
    wp = _weights(weights, T, J, ys)
    dp, ldr = _rows(residual, T, H, "residual", ys) if residual is not None else (None, 0)
    with _On(ys.device, stream) as on:
        if out is None:
            out = torch.empty((T, H), dtype=ys.dtype, device=ys.device)
        yp, ldy = _rows(out, T, H, "out", ys)
        _check(load_library().expert_combine(kind, T, J, H, rp, wp, sp, lds, dp, ldr, yp, ldy, on.stream.cuda_stream),
               "expert_combine")
    return out


def expert_gather_backward(dxs, rows, stream=None):
    """dx of expert_gather: the sum of each token's rows of dxs."""
    return expert_combine(dxs, rows, stream=stream)


def expert_combine_backward(dy, ys, rows, weights, offsets, need_dweights=True, stream=None):
    """(dys, dweights) of expert_combine (the residual's gradient is dy itself):
    dys[rows[t, j]] = weights[t, j] * dy[t], 0 in the places in no use, and
    dweights[t, j] = dy[t] . ys[rows[t, j]], float32, 0 for a dropped choice."""
    import torch
    kind = _type_of(dy, "dy")
    if dy.dim() != 2:
        raise ValueError(f"dy must be 2-D, got {tuple(dy.shape)}")
    T, H = dy.shape
    gp, lddy = _rows(dy, T, H, "dy")
    J, E, rp, op = _order(rows, offsets, T, dy)
    wp = _weights(weights, T, J, dy)
    sp, lds = _rows(ys, T * J, H, "ys", dy) if need_dweights else (None, 0)
    with _On(dy.device, stream) as on:
        dys = torch.empty((T * J, H), dtype=dy.dtype, device=dy.device)
        dweights = torch.empty((T, J), dtype=torch.float32, device=dy.device) if need_dweights else None
        _check(load_library().expert_combine_backward(kind, T, J, H, E, rp, op, wp, gp, lddy, sp, lds, dys.data_ptr(),
                                                      max(H, 1), dweights.data_ptr() if need_dweights else None,
                                                      on.stream.cuda_stream), "expert_combine_backward")
    return dys, dweights
