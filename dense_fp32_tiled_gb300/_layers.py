"""Layer operators on torch tensors: argument marshalling for include/linear.h,
include/experts.h, include/norm.h and include/cross_entropy.h.  As in
``_binding``, every arithmetic step runs in the CUDA library; PyTorch supplies
device memory, strides and the current stream.

Every function runs on ``stream`` (a torch.cuda.Stream) or the current one, is
asynchronous, and allocates what it returns on that stream.  Tensors of one
call share a device and a type (float32, bfloat16 or float16).  Wrong shapes
and types raise ValueError and TypeError before anything is launched; a
status of the library raises SgemmError.
"""
from __future__ import annotations

import ctypes
import operator
from contextlib import nullcontext

from ._binding import SGEMM_OK, SgemmError, load_library

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
SCORINGS = {"softmax": 0, "sigmoid": 1}

# What these calls launch is short (a decoding step's product takes a few
# microseconds), so calls on the current device and stream whose arguments are
# as they should be go through an extension (csrc/fast_call.c) that takes the
# same steps without the interpreter.  It answers NotImplemented to anything
# else, which the functions below then serve or refuse, and a status of the
# library as a number.
torch = None
_lib = None
_types = {}
_raw_stream = None
_fast = None


def _load():
    global torch, _lib, _raw_stream, _fast
    if _lib is None:
        import torch as _torch
        torch = _torch
        _types.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
        _raw_stream = torch._C._cuda_getCurrentRawStream
        _lib = load_library()
        try:
            from . import _fast_call
        except ImportError:  # built without Python's headers
            return _lib
        names = [f for op in ("linear_forward", "linear_backward", "expert_linear_forward", "expert_linear_backward",
                              "expert_sort") for f in (op, op + "_workspace_size")]
        names += ["expert_gather", "expert_combine", "expert_combine_backward"]
        _fast_call.bind({n: ctypes.cast(getattr(_lib, n), ctypes.c_void_p).value for n in names},
                        bound(torch, _raw_stream, torch._C._cuda_getDevice))
        names = ["layer_norm_forward", "expert_choose", "expert_choose_backward"]
        names += [f for op in ("layer_norm_backward", "linear_cross_entropy_forward", "linear_cross_entropy_backward")
                  for f in (op, op + "_workspace_size")]
        _fast_call.bind_more({n: ctypes.cast(getattr(_lib, n), ctypes.c_void_p).value for n in names}, SCORINGS)
        _fast = _fast_call
    return _lib


def bound(torch, raw_stream, get_device):
    """What the extension's calls need of torch."""
    return (torch.Tensor, torch.empty, raw_stream, get_device, ACTIVATIONS, (torch.float32, torch.bfloat16, torch.float16),
            torch.int32, torch.int64, torch.uint8)


def _type_of(t, name):
    kind = _types.get(getattr(t, "dtype", None))
    if kind is None or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor of float32, bfloat16 or float16")
    return kind


def _fits(*sizes):
    """The C functions' sizes are 32-bit."""
    if any(abs(n) > 0x7fffffff for n in sizes):
        raise ValueError(f"sizes must be below 2**31, got {sizes}")


def _alike(t, dtype, device, name):
    if getattr(t, "dtype", None) is not dtype or t.get_device() != device:
        raise TypeError(f"{name} must be a {dtype} tensor on cuda:{device}")


def _rows(t, rows, cols, dtype, device, name):
    """(address, row stride) of a row-major rows x cols tensor."""
    if getattr(t, "dtype", None) is not dtype or t.get_device() != device:
        _alike(t, dtype, device, name)
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must have shape ({rows}, {cols}), got {tuple(t.shape)}")
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{name} must be row-major with unit column stride")
    if ld < cols or ld < 1:
        if rows > 1:
            raise ValueError(f"{name} has overlapping rows")
        ld = max(cols, 1)
    return t.data_ptr(), ld


def _vector(t, shape, dtype, device, name):
    if t is None:
        return None
    _alike(t, dtype, device, name)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {shape}, got {tuple(t.shape)}")
    return t.data_ptr()


def _weight(w, K, dtype, device, name):
    """(address, stride, order, expert stride) of (..., K, N) with either of the last two contiguous."""
    _alike(w, dtype, device, name)
    if w.shape[-2] != K:
        raise ValueError(f"{name} must have {K} inputs in its last but one dimension, got {tuple(w.shape)}")
    N = w.shape[-1]
    strides = w.stride()
    sk, sn = strides[-2:]
    expert = strides[0] if len(strides) == 3 and w.shape[0] > 1 else 0
    if (sn == 1 or N == 1) and (sk >= N or K <= 1):
        return w.data_ptr(), (sk if K > 1 else max(sk, N, 1)), 0, expert
    if (sk == 1 or K == 1) and (sn >= K or N <= 1):
        return w.data_ptr(), (sn if N > 1 else max(sn, K, 1)), 1, expert
    raise ValueError(f"{name} must have one of its last two dimensions contiguous, its rows apart")


def _int32(t, shape, device, name):
    if getattr(t, "dtype", None) is not torch.int32 or t.get_device() != device:
        raise TypeError(f"{name} must be an int32 tensor on cuda:{device}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {shape}, got {tuple(t.shape)}")
    return t.data_ptr()


def _grouped(offsets):
    if offsets is None:
        raise ValueError("offsets are needed (linear is the product without them)")


_NOWHERE = nullcontext()


def _on(device, stream):
    """The context in which a call allocates and launches: the device and stream it is for."""
    if stream is not None:
        if stream.device.index != device:
            raise ValueError(f"stream is on cuda:{stream.device.index}, the tensors on cuda:{device}")
        return torch.cuda.stream(stream)
    if torch.cuda.current_device() != device:
        return torch.cuda.device(device)
    return _NOWHERE


def _scratch(nbytes, device):
    """Scratch of one call, or None.  It is the call's own: allocated with the
    call's stream current and given back to torch's allocator when all its
    kernels are enqueued, which hands it on in the order of that stream only.
    So no two threads' calls have the same at a time, and a captured graph's
    is memory of that graph."""
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _act(name):
    act = ACTIVATIONS.get(name)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {name!r}")
    return act


def _check(st, what):
    if st != SGEMM_OK:
        raise SgemmError(st, what)


def _answer(r, what):
    if type(r) is int:
        raise SgemmError(r, what)
    return r


# ---- the product with its epilogue ---------------------------------------------
def linear(x, w, bias=None, residual=None, activation="none", preact=None, out=None, stream=None):
    """act(x @ w + bias) + residual.

    x is (M, K), row-major with any row stride; w is (K, N) in either memory
    order (``weight.t()`` of an (N, K) weight is read as it is); bias is (N,);
    residual and out are (M, N).  ``preact``, an (M, N) tensor, receives
    x @ w + bias for linear_backward.  ``out`` may be ``residual`` itself.
    """
    if stream is None and _fast is not None:
        r = _fast.forward(x, w, None, bias, residual, activation, preact, out)
        if r is not NotImplemented:
            return _answer(r, "linear_forward")
    return _forward(x, w, None, bias, residual, activation, preact, out, stream)


def expert_linear(x, w, offsets, bias=None, residual=None, activation="none", preact=None, out=None, stream=None):
    """The same product over rows sorted by expert: rows offsets[e] to
    offsets[e + 1] of x (R, K) meet w[e] and bias[e] of w (E, K, N) and bias
    (E, N).  offsets is int32 (E + 1,) on the device, as expert_sort makes it,
    and is not read on the host.  Rows of no expert give 0."""
    _grouped(offsets)
    if stream is None and _fast is not None:
        r = _fast.forward(x, w, offsets, bias, residual, activation, preact, out)
        if r is not NotImplemented:
            return _answer(r, "expert_linear_forward")
    return _forward(x, w, offsets, bias, residual, activation, preact, out, stream)


def _forward(x, w, offsets, bias, residual, activation, preact, out, stream):
    lib = _lib or _load()
    kind, act = _type_of(x, "x"), _act(activation)
    grouped = offsets is not None
    if x.dim() != 2 or w.dim() != 2 + grouped:
        raise ValueError(f"x must be 2-D and w {2 + grouped}-D, got {tuple(x.shape)} and {tuple(w.shape)}")
    (M, K), dtype, dev = x.shape, x.dtype, x.get_device()
    xp, ldx = _rows(x, M, K, dtype, dev, "x")
    wp, ldw, order, step = _weight(w, K, dtype, dev, "w")
    N = w.shape[-1]
    _fits(M, N, K)
    rp, ldr = _rows(residual, M, N, dtype, dev, "residual") if residual is not None else (None, 0)
    zp, ldz = _rows(preact, M, N, dtype, dev, "preact") if preact is not None else (None, 0)
    if grouped:
        E = w.shape[0]
        op = _int32(offsets, (E + 1,), dev, "offsets")
    bp = _vector(bias, (E, N) if grouped else (N,), dtype, dev, "bias")
    with _on(dev, stream):
        if out is None:
            out = torch.empty((M, N), dtype=dtype, device=x.device)
            yp, ldy = out.data_ptr(), N or 1
        else:
            yp, ldy = _rows(out, M, N, dtype, dev, "out")
        raw = _raw_stream(dev)
        nbytes, ws, wsp = 0, None, None
        if kind == 0 or (xp | wp) & 15 or (ldx | ldw | step) & 7:
            nbytes = (lib.expert_linear_forward_workspace_size(kind, M, N, K, E, xp, ldx, wp, ldw, step, order) if grouped
                      else lib.linear_forward_workspace_size(kind, M, N, K, xp, ldx, wp, ldw, order))
            ws = _scratch(nbytes, x.device)
            wsp = ws.data_ptr() if nbytes else None
        if grouped:
            st = lib.expert_linear_forward(kind, M, N, K, E, op, xp, ldx, wp, ldw, step, order, bp, rp, ldr, act, zp, ldz,
                                           yp, ldy, wsp, nbytes, raw)
        else:
            st = lib.linear_forward(kind, M, N, K, xp, ldx, wp, ldw, order, bp, rp, ldr, act, zp, ldz, yp, ldy, wsp, nbytes,
                                    raw)
    if st:
        _check(st, "expert_linear_forward" if grouped else "linear_forward")
    return out


def linear_backward(dy, x, w, preact=None, activation="none", need_dx=True, need_dw=True, need_dbias=True, stream=None):
    """(dx, dw, dbias) of linear for the gradient dy of its result (that of the
    residual is dy itself).  preact is what linear saved, needed unless the
    activation is "none".  dw has the memory order of w; what is not needed is None."""
    if stream is None and _fast is not None:
        r = _fast.backward(dy, x, w, None, preact, activation, need_dx, need_dw, need_dbias)
        if r is not NotImplemented:
            return _answer(r, "linear_backward")
    return _backward(dy, x, w, None, preact, activation, need_dx, need_dw, need_dbias, stream)


def expert_linear_backward(dy, x, w, offsets, preact=None, activation="none", need_dx=True, need_dw=True,
                           need_dbias=True, stream=None):
    """(dx, dw, dbias) of expert_linear.  Rows of no expert have a dx of 0, experts without rows a dw and dbias of 0."""
    _grouped(offsets)
    if stream is None and _fast is not None:
        r = _fast.backward(dy, x, w, offsets, preact, activation, need_dx, need_dw, need_dbias)
        if r is not NotImplemented:
            return _answer(r, "expert_linear_backward")
    return _backward(dy, x, w, offsets, preact, activation, need_dx, need_dw, need_dbias, stream)


def _backward(dy, x, w, offsets, preact, activation, need_dx, need_dw, need_dbias, stream):
    lib = _lib or _load()
    kind, act = _type_of(x, "x"), _act(activation)
    grouped = offsets is not None
    if x.dim() != 2 or w.dim() != 2 + grouped:
        raise ValueError(f"x must be 2-D and w {2 + grouped}-D, got {tuple(x.shape)} and {tuple(w.shape)}")
    if (preact is None) != (act == 0):
        raise ValueError("preact is needed with an activation, and only then")
    (M, K), dtype, dev = x.shape, x.dtype, x.get_device()
    N = w.shape[-1]
    _fits(M, N, K)
    gp, lddy = _rows(dy, M, N, dtype, dev, "dy")
    xp, ldx = _rows(x, M, K, dtype, dev, "x")
    wp, ldw, order, step = _weight(w, K, dtype, dev, "w")
    zp, ldz = _rows(preact, M, N, dtype, dev, "preact") if preact is not None else (None, 0)
    lead = ()
    if grouped:
        E = w.shape[0]
        lead = (E,)
        op = _int32(offsets, (E + 1,), dev, "offsets")
    dx = dw = dbias = hp = vp = bp = None
    ldh, ldv, stepv = K or 1, (K if order else N) or 1, K * N
    with _on(dev, stream):
        if need_dx:
            dx = torch.empty((M, K), dtype=dtype, device=x.device)
            hp = dx.data_ptr()
        if need_dw:
            dw = torch.empty(lead + ((N, K) if order else (K, N)), dtype=dtype, device=x.device)
            vp = dw.data_ptr()
            if order:
                dw = dw.transpose(-1, -2)
        if need_dbias:
            dbias = torch.empty(lead + (N,), dtype=dtype, device=x.device)
            bp = dbias.data_ptr()
        raw = _raw_stream(dev)
        if grouped:
            nbytes = lib.expert_linear_backward_workspace_size(kind, M, N, K, E, gp, lddy, xp, ldx, wp, ldw, step, order,
                                                               act, need_dx, need_dw, need_dbias)
            ws = _scratch(nbytes, x.device)
            st = lib.expert_linear_backward(kind, M, N, K, E, op, gp, lddy, xp, ldx, wp, ldw, step, order, zp, ldz, act, hp,
                                            ldh, vp, ldv, stepv, bp, ws.data_ptr() if nbytes else None, nbytes, raw)
        else:
            nbytes = lib.linear_backward_workspace_size(kind, M, N, K, gp, lddy, xp, ldx, wp, ldw, order, act, need_dx,
                                                        need_dw, need_dbias)
            ws = _scratch(nbytes, x.device)
            st = lib.linear_backward(kind, M, N, K, gp, lddy, xp, ldx, wp, ldw, order, zp, ldz, act, hp, ldh, vp, ldv, bp,
                                     ws.data_ptr() if nbytes else None, nbytes, raw)
    if st:
        _check(st, "expert_linear_backward" if grouped else "linear_backward")
    return dx, dw, dbias


def linear_timeouts() -> int:
    """1 if a kernel of the layer products gave up a wait since the library was loaded, else 0."""
    n = ctypes.c_uint()
    _check(load_library().linear_timeouts(ctypes.byref(n)), "linear_timeouts")
    return n.value


# ---- the loss of a head ----------------------------------------------------------
def _integers(t, shape, device, name):
    """(address, bytes of a value) of a contiguous int32 or int64 tensor."""
    dtype = getattr(t, "dtype", None)
    if (dtype is not torch.int32 and dtype is not torch.int64) or t.get_device() != device:
        raise TypeError(f"{name} must be an int32 or int64 tensor on cuda:{device}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {shape}, got {tuple(t.shape)}")
    return t.data_ptr(), 4 if dtype is torch.int32 else 8


def _head(x, w, targets):
    kind = _type_of(x, "x")
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError(f"x and w must be 2-D, got {tuple(x.shape)} and {tuple(w.shape)}")
    (M, K), dtype, dev = x.shape, x.dtype, x.get_device()
    xp, ldx = _rows(x, M, K, dtype, dev, "x")
    wp, ldw, order, _ = _weight(w, K, dtype, dev, "w")
    N = w.shape[1]
    _fits(M, N, K)
    tp, width = _integers(targets, (M,), dev, "targets")
    return kind, M, N, K, xp, ldx, wp, ldw, order, tp, width


def linear_cross_entropy(x, w, targets, stream=None):
    """(loss, lse): each row's -log softmax(x @ w)[target] and log of its sum of
    exponentials, float32 (M,), without x @ w in memory.

    x is (M, K), row-major with any row stride; w is (K, N) in either memory
    order; targets is int32 or int64 (M,).  A target outside 0 .. N - 1 (a
    padded token's -100) gives a loss of 0.
    """
    if stream is None and _fast is not None:
        r = _fast.cross_entropy(x, w, targets)
        if r is not NotImplemented:
            return _answer(r, "linear_cross_entropy_forward")
    lib = _lib or _load()
    kind, M, N, K, xp, ldx, wp, ldw, order, tp, width = _head(x, w, targets)
    with _on(x.get_device(), stream):
        loss = torch.empty((M,), dtype=torch.float32, device=x.device)
        lse = torch.empty((M,), dtype=torch.float32, device=x.device)
        nbytes = lib.linear_cross_entropy_forward_workspace_size(kind, M, N, K, xp, ldx, wp, ldw, order)
        ws = _scratch(nbytes, x.device)
        st = lib.linear_cross_entropy_forward(kind, M, N, K, xp, ldx, wp, ldw, order, tp, width, loss.data_ptr(),
                                              lse.data_ptr(), ws.data_ptr() if nbytes else None, nbytes,
                                              _raw_stream(x.get_device()))
    if st:
        _check(st, "linear_cross_entropy_forward")
    return loss, lse


def linear_cross_entropy_backward(dloss, x, w, targets, lse, dlse=None, need_dx=True, need_dw=True, stream=None):
    """(dx, dw) of linear_cross_entropy for the gradients of its losses and (dlse,
    None for none) of its log sums, float32 (M,); lse is what it returned.  dw
    has the memory order of w; what is not needed is None.  In the 16-bit types
    the logits' gradients are rounded to them, as fractions of the largest, before
    the two products."""
    if stream is None and _fast is not None:
        r = _fast.cross_entropy_backward(dloss, x, w, targets, lse, dlse, need_dx, need_dw)
        if r is not NotImplemented:
            return _answer(r, "linear_cross_entropy_backward")
    lib = _lib or _load()
    kind, M, N, K, xp, ldx, wp, ldw, order, tp, width = _head(x, w, targets)
    dev = x.get_device()
    if lse is None:
        raise ValueError("lse is needed (linear_cross_entropy returns it)")
    gp, ep = _vector(dloss, (M,), torch.float32, dev, "dloss"), _vector(dlse, (M,), torch.float32, dev, "dlse")
    lp = _vector(lse, (M,), torch.float32, dev, "lse")
    dx = dw = hp = vp = None
    with _on(dev, stream):
        if need_dx:
            dx = torch.empty((M, K), dtype=x.dtype, device=x.device)
            hp = dx.data_ptr()
        if need_dw:
            dw = torch.empty((N, K) if order else (K, N), dtype=x.dtype, device=x.device)
            vp = dw.data_ptr()
            if order:
                dw = dw.transpose(0, 1)
        nbytes = lib.linear_cross_entropy_backward_workspace_size(kind, M, N, K, xp, ldx, wp, ldw, order, bool(need_dx), bool(need_dw))
        ws = _scratch(nbytes, x.device)
        st = lib.linear_cross_entropy_backward(kind, M, N, K, gp, ep, xp, ldx, wp, ldw, order, tp, width, lp, hp, K or 1, vp,
                                               (K if order else N) or 1, ws.data_ptr() if nbytes else None, nbytes,
                                               _raw_stream(dev))
    if st:
        _check(st, "linear_cross_entropy_backward")
    return dx, dw


# ---- layer norm ------------------------------------------------------------------
def layer_norm(x, weight=None, bias=None, eps=1e-5, stats=None, out=None, stream=None):
    """(x - mean) / sqrt(variance + eps) * weight + bias over the rows of x.

    x is (M, N), row-major with any row stride; weight and bias are (N,), None
    for 1 and 0; out is (M, N).  ``stats``, a float32 (M, 2) tensor, receives
    each row's mean and 1 / sqrt(variance + eps) for layer_norm_backward.
    """
    if stream is None and _fast is not None:
        r = _fast.norm(x, weight, bias, eps, stats, out)
        if r is not NotImplemented:
            return _answer(r, "layer_norm_forward")
    lib = _lib or _load()
    kind = _type_of(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got {tuple(x.shape)}")
    (M, N), dtype, dev = x.shape, x.dtype, x.get_device()
    _fits(M, N)
    xp, ldx = _rows(x, M, N, dtype, dev, "x")
    wp, bp = _vector(weight, (N,), dtype, dev, "weight"), _vector(bias, (N,), dtype, dev, "bias")
    sp = _vector(stats, (M, 2), torch.float32, dev, "stats")
    with _on(dev, stream):
        if out is None:
            out = torch.empty((M, N), dtype=dtype, device=x.device)
        yp, ldy = _rows(out, M, N, dtype, dev, "out")
        st = lib.layer_norm_forward(kind, M, N, xp, ldx, wp, bp, eps, sp, yp, ldy, _raw_stream(dev))
    if st:
        _check(st, "layer_norm_forward")
    return out


def layer_norm_backward(dy, x, weight, stats, need_dx=True, need_dweight=True, need_dbias=True, stream=None):
    """(dx, dweight, dbias) of layer_norm for the gradient dy of its result.
    stats is what layer_norm saved; weight may be None (all 1).  What is not
    needed is None."""
    if stream is None and _fast is not None:
        r = _fast.norm_backward(dy, x, weight, stats, need_dx, need_dweight, need_dbias)
        if r is not NotImplemented:
            return _answer(r, "layer_norm_backward")
    lib = _lib or _load()
    kind = _type_of(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got {tuple(x.shape)}")
    (M, N), dtype, dev = x.shape, x.dtype, x.get_device()
    _fits(M, N)
    gp, lddy = _rows(dy, M, N, dtype, dev, "dy")
    xp, ldx = _rows(x, M, N, dtype, dev, "x")
    wp = _vector(weight, (N,), dtype, dev, "weight")
    if stats is None:
        raise ValueError("stats are needed (layer_norm saves them)")
    sp = _vector(stats, (M, 2), torch.float32, dev, "stats")
    dx = dweight = dbias = None
    with _on(dev, stream):
        if need_dx:
            dx = torch.empty((M, N), dtype=dtype, device=x.device)
        if need_dweight:
            dweight = torch.empty((N,), dtype=dtype, device=x.device)
        if need_dbias:
            dbias = torch.empty((N,), dtype=dtype, device=x.device)
        nbytes = lib.layer_norm_backward_workspace_size(M, N, bool(need_dweight), bool(need_dbias))
        ws = _scratch(nbytes, x.device)
        st = lib.layer_norm_backward(kind, M, N, gp, lddy, xp, ldx, wp, sp, dx.data_ptr() if need_dx else None, N or 1,
                                     dweight.data_ptr() if need_dweight else None, dbias.data_ptr() if need_dbias else None,
                                     ws.data_ptr() if nbytes else None, nbytes, _raw_stream(dev))
    if st:
        _check(st, "layer_norm_backward")
    return dx, dweight, dbias


# ---- tokens to their experts and back --------------------------------------------
def _scoring(name):
    scoring = SCORINGS.get(name)
    if scoring is None:
        raise ValueError(f"scoring must be one of {', '.join(SCORINGS)}, got {name!r}")
    return scoring


def expert_choose(logits, choices, bias=None, scoring="softmax", groups=1, kept_groups=1, group_top=1, renormalize=True,
                  scale=1.0, stream=None):
    """(chosen, weights): each token's experts from a router's logits (T, E), for
    expert_sort and expert_combine.

    Scores are softmax or sigmoid of the logits.  The ``choices`` experts with
    the largest score + bias (bias: float32 (E,) or None) are chosen, in falling
    order, of equal ones the lowest; with ``groups`` > 1 only those of the
    ``kept_groups`` groups (of E / groups experts in a row) whose ``group_top``
    (1 or 2) best have the largest sum.  chosen is int32 (T, choices); weights,
    float32, are scale times the chosen scores, divided by their sum if
    ``renormalize``.  Experts with a logit of -inf are never chosen; places left
    over are -1 (which expert_sort drops), their weights 0.  A token with a NaN
    among its logits chooses none, and its weights are NaN.
    """
    if stream is None and _fast is not None:
        r = _fast.choose(logits, choices, bias, scoring, groups, kept_groups, group_top, renormalize, scale)
        if r is not NotImplemented:
            return _answer(r, "expert_choose")
    lib = _lib or _load()
    kind, how = _type_of(logits, "logits"), _scoring(scoring)
    if logits.dim() != 2:
        raise ValueError(f"logits must be 2-D, got {tuple(logits.shape)}")
    (T, E), dtype, dev = logits.shape, logits.dtype, logits.get_device()
    J, groups, kept_groups, group_top = (operator.index(n) for n in (choices, groups, kept_groups, group_top))
    _fits(T, E, J, groups, kept_groups, group_top)
    lp, ldl = _rows(logits, T, E, dtype, dev, "logits")
    bp = _vector(bias, (E,), torch.float32, dev, "bias")
    with _on(dev, stream):
        chosen = torch.empty((T, max(J, 0)), dtype=torch.int32, device=logits.device)
        weights = torch.empty((T, max(J, 0)), dtype=torch.float32, device=logits.device)
        st = lib.expert_choose(kind, T, E, J, lp, ldl, bp, how, groups, kept_groups, group_top, bool(renormalize), scale,
                               chosen.data_ptr(), weights.data_ptr(), _raw_stream(dev))
    if st:
        _check(st, "expert_choose")
    return chosen, weights


def expert_choose_backward(dweights, logits, chosen, scoring="softmax", renormalize=True, scale=1.0, stream=None):
    """The gradient of the logits, in their type, from that of expert_choose's
    weights; chosen, scoring, renormalize and scale as there (the bias has none)."""
    if stream is None and _fast is not None:
        r = _fast.choose_backward(dweights, logits, chosen, scoring, renormalize, scale)
        if r is not NotImplemented:
            return _answer(r, "expert_choose_backward")
    lib = _lib or _load()
    kind, how = _type_of(logits, "logits"), _scoring(scoring)
    if logits.dim() != 2 or getattr(chosen, "ndim", 2) != 2:
        raise ValueError(f"logits and chosen must be 2-D, got {tuple(logits.shape)} and {tuple(chosen.shape)}")
    (T, E), J, dtype, dev = logits.shape, chosen.shape[1], logits.dtype, logits.get_device()
    _fits(T, E, J)
    lp, ldl = _rows(logits, T, E, dtype, dev, "logits")
    cp = _int32(chosen, (T, J), dev, "chosen")
    if dweights is None:
        raise ValueError("dweights are needed")
    gp = _vector(dweights, (T, J), torch.float32, dev, "dweights")
    with _on(dev, stream):
        dlogits = torch.empty((T, E), dtype=dtype, device=logits.device)
        st = lib.expert_choose_backward(kind, T, E, J, gp, cp, lp, ldl, how, bool(renormalize), scale, dlogits.data_ptr(),
                                        E or 1, _raw_stream(dev))
    if st:
        _check(st, "expert_choose_backward")
    return dlogits


def expert_sort(choices, experts, stream=None):
    """(rows, offsets): choices is int32 or int64 (T, J), the experts of each
    token (one outside 0 .. experts - 1 is dropped).  rows, int32 (T, J), is
    each choice's place among all T*J sorted by expert, then token and choice,
    or -1; places offsets[e] to offsets[e + 1] belong to expert e."""
    if stream is None and _fast is not None:
        r = _fast.sort(choices, experts)
        if r is not NotImplemented:
            return _answer(r, "expert_sort")
    lib = _lib or _load()
    dtype = getattr(choices, "dtype", None)
    if dtype is torch.int32:
        width = 4
    elif dtype is torch.int64:
        width = 8
    else:
        raise TypeError("choices must be a CUDA tensor of int32 or int64")
    if not choices.is_cuda:
        raise TypeError("choices must be a CUDA tensor of int32 or int64")
    if choices.dim() != 2 or not choices.is_contiguous():
        raise ValueError(f"choices must be contiguous with shape (tokens, choices), got {tuple(choices.shape)}")
    (T, J), E, dev = choices.shape, int(experts), choices.get_device()
    _fits(T, J, E)
    with _on(dev, stream):
        rows = torch.empty((T, J), dtype=torch.int32, device=choices.device)
        offsets = torch.empty((max(E, 0) + 1,), dtype=torch.int32, device=choices.device)
        raw = _raw_stream(dev)
        nbytes = lib.expert_sort_workspace_size(T, J, E)
        ws = _scratch(nbytes, choices.device)
        st = lib.expert_sort(T, J, E, choices.data_ptr(), width, rows.data_ptr(), offsets.data_ptr(),
                             ws.data_ptr() if nbytes else None, nbytes, raw)
    if st:
        _check(st, "expert_sort")
    return rows, offsets


def _order(rows, offsets, T, dev):
    """(choices, experts, address of rows, address of offsets)."""
    if rows.dim() != 2 or offsets is not None and offsets.dim() != 1:
        raise ValueError("rows must be 2-D and offsets 1-D")
    J, E = rows.shape[1], 0
    op = None
    if offsets is not None:
        E = offsets.shape[0] - 1
        op = _int32(offsets, (E + 1,), dev, "offsets")
    _fits(J, E)
    return J, E, _int32(rows, (T, J), dev, "rows"), op


def expert_gather(x, rows, offsets, out=None, stream=None):
    """The token rows in expert order: out[rows[t, j]] = x[t], (T*J, H); places in no use are 0."""
    if stream is None and _fast is not None:
        r = _fast.gather(x, rows, offsets, out)
        if r is not NotImplemented:
            return _answer(r, "expert_gather")
    lib = _lib or _load()
    kind = _type_of(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got {tuple(x.shape)}")
    (T, H), dtype, dev = x.shape, x.dtype, x.get_device()
    _fits(T, H)
    xp, ldx = _rows(x, T, H, dtype, dev, "x")
    J, E, rp, op = _order(rows, offsets, T, dev)
    with _on(dev, stream):
        if out is None:
            out = torch.empty((T * J, H), dtype=dtype, device=x.device)
        sp, lds = _rows(out, T * J, H, dtype, dev, "out")
        st = lib.expert_gather(kind, T, J, H, E, rp, op, xp, ldx, sp, lds, _raw_stream(dev))
    if st:
        _check(st, "expert_gather")
    return out


def expert_combine(ys, rows, weights=None, residual=None, out=None, stream=None):
    """Each token's sum over its choices: residual[t] + sum_j weights[t, j] * ys[rows[t, j]].
    weights is float32 (T, J); None weighs all by 1.  Dropped choices add nothing."""
    if stream is None and _fast is not None:
        r = _fast.combine(ys, rows, weights, residual, out)
        if r is not NotImplemented:
            return _answer(r, "expert_combine")
    lib = _lib or _load()
    kind = _type_of(ys, "ys")
    if ys.dim() != 2 or rows.dim() != 2:
        raise ValueError(f"ys and rows must be 2-D, got {tuple(ys.shape)} and {tuple(rows.shape)}")
    T, H, dtype, dev = rows.shape[0], ys.shape[1], ys.dtype, ys.get_device()
    _fits(T, H)
    J, _, rp, _ = _order(rows, None, T, dev)
    sp, lds = _rows(ys, T * J, H, dtype, dev, "ys")
    wp = _vector(weights, (T, J), torch.float32, dev, "weights")
    dp, ldr = _rows(residual, T, H, dtype, dev, "residual") if residual is not None else (None, 0)
    with _on(dev, stream):
        if out is None:
            out = torch.empty((T, H), dtype=dtype, device=ys.device)
        yp, ldy = _rows(out, T, H, dtype, dev, "out")
        st = lib.expert_combine(kind, T, J, H, rp, wp, sp, lds, dp, ldr, yp, ldy, _raw_stream(dev))
    if st:
        _check(st, "expert_combine")
    return out


def expert_gather_backward(dxs, rows, stream=None):
    """dx of expert_gather: the sum of each token's rows of dxs."""
    return expert_combine(dxs, rows, stream=stream)


def expert_combine_backward(dy, ys, rows, weights, offsets, need_dweights=True, stream=None):
    """(dys, dweights) of expert_combine (the residual's gradient is dy itself):
    dys[rows[t, j]] = weights[t, j] * dy[t], 0 in the places in no use, and
    dweights[t, j] = dy[t] . ys[rows[t, j]], float32, 0 for a dropped choice."""
    if stream is None and _fast is not None:
        r = _fast.combine_backward(dy, ys, rows, weights, offsets, need_dweights)
        if r is not NotImplemented:
            return _answer(r, "expert_combine_backward")
    lib = _lib or _load()
    kind = _type_of(dy, "dy")
    if dy.dim() != 2:
        raise ValueError(f"dy must be 2-D, got {tuple(dy.shape)}")
    (T, H), dtype, dev = dy.shape, dy.dtype, dy.get_device()
    _fits(T, H)
    gp, lddy = _rows(dy, T, H, dtype, dev, "dy")
    J, E, rp, op = _order(rows, offsets, T, dev)
    wp = _vector(weights, (T, J), torch.float32, dev, "weights")
    sp, lds = _rows(ys, T * J, H, dtype, dev, "ys") if need_dweights else (None, 0)
    dweights = None
    with _on(dev, stream):
        dys = torch.empty((T * J, H), dtype=dtype, device=dy.device)
        if need_dweights:
            dweights = torch.empty((T, J), dtype=torch.float32, device=dy.device)
        st = lib.expert_combine_backward(kind, T, J, H, E, rp, op, wp, gp, lddy, sp, lds, dys.data_ptr(), H or 1,
                                         dweights.data_ptr() if need_dweights else None, _raw_stream(dev))
    if st:
        _check(st, "expert_combine_backward")
    return dys, dweights
