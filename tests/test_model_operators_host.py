"""Refusals of expert_choose, layer_norm and linear_cross_entropy, all before any
CUDA call, and what their calls do around their launches (CPU only)."""
import gc

import pytest

import dense_fp32_tiled_gb300 as sg
from dense_fp32_tiled_gb300 import build as sg_build

A, B, C, D, E_, F_, G, WS = (0x100000 * (i + 1) for i in range(8))  # never dereferenced
BF16, F32, F16 = 1, 0, 2


@pytest.fixture(scope="module")
def lib():
    sg_build.build()
    return sg.load_library()


def choose(lib, type=F32, T=4, E=16, J=2, l=A, ld=16, bias=None, how=0, groups=1, kept=1, top=1, renorm=1, scale=1.0, chosen=C, w=D):
    return lib.expert_choose(type, T, E, J, l, ld, bias, how, groups, kept, top, renorm, scale, chosen, w, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), -7), (dict(how=2), -7), (dict(how=-1), -7), (dict(groups=0), -7), (dict(groups=3), -7), (dict(groups=33, E=33, ld=33), -7),
    (dict(groups=4, kept=5), -7), (dict(groups=4, kept=0), -7), (dict(groups=4, top=3), -7), (dict(groups=4, top=0), -7),
    (dict(T=-1), -1), (dict(E=0), -1), (dict(E=1025, ld=1025), -1), (dict(J=-1), -1), (dict(J=17), -1), (dict(E=100, ld=100, J=65), -1),
    (dict(T=2 ** 31 - 1), -1), (dict(T=2 ** 30, J=4), -1), (dict(ld=15), -2), (dict(l=None), -3), (dict(chosen=None), -3), (dict(w=None), -3),
    (dict(l=A + 2), -7), (dict(bias=B + 2), -7), (dict(chosen=C + 2), -7), (dict(w=D + 1), -7), (dict(type=BF16, l=A + 1), -7),
    (dict(chosen=A + 64), -4), (dict(w=A), -4), (dict(bias=B, chosen=B + 4), -4), (dict(w=C + 4), -4),
    (dict(T=0, l=None, chosen=None, w=None), 0), (dict(J=0, chosen=None, w=None), 0),
])
def test_choose_refusals(lib, kw, code):
    assert choose(lib, **kw) == code


def choose_back(lib, type=F32, T=4, E=16, J=2, g=B, chosen=C, l=A, ld=16, how=0, renorm=1, scale=1.0, d=D, ldd=16):
    return lib.expert_choose_backward(type, T, E, J, g, chosen, l, ld, how, renorm, scale, d, ldd, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=-1), -7), (dict(how=3), -7), (dict(E=2000, ld=2000, ldd=2000), -1), (dict(ld=15), -2), (dict(ldd=15), -2), (dict(g=None), -3),
    (dict(chosen=None), -3), (dict(l=None), -3), (dict(d=None), -3), (dict(d=A), -4), (dict(d=B - 64), -4), (dict(d=C - 4), -4),
    (dict(d=D + 2), -7), (dict(T=0), 0),
])
def test_choose_backward_refusals(lib, kw, code):
    assert choose_back(lib, **kw) == code


def norm(lib, type=BF16, M=4, N=16, x=A, ldx=16, w=B, b=C, eps=1e-5, stats=D, y=E_, ldy=16):
    return lib.layer_norm_forward(type, M, N, x, ldx, w, b, eps, stats, y, ldy, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), -7), (dict(M=-1), -1), (dict(N=-1), -1), (dict(M=2 ** 31 - 1), -1), (dict(N=2 ** 31 - 1, ldx=2 ** 31, ldy=2 ** 31), -1),
    (dict(eps=-1e-9), -7), (dict(eps=float("nan")), -7), (dict(eps=float("inf")), -7), (dict(ldx=15), -2), (dict(ldy=15), -2),
    (dict(N=0, ldx=0), -2), (dict(x=None), -3), (dict(y=None), -3), (dict(x=A + 1), -7), (dict(w=B + 1), -7), (dict(b=C + 1), -7),
    (dict(stats=D + 2), -7), (dict(y=E_ + 1), -7), (dict(y=A), -4), (dict(y=A + 126), -4), (dict(y=B), -4), (dict(stats=C), -4),
    (dict(stats=E_ + 4), -4), (dict(M=0, x=None, y=None), 0), (dict(N=0, x=None, y=None, stats=None), 0),
])
def test_norm_refusals(lib, kw, code):
    assert norm(lib, **kw) == code


def norm_back(lib, type=BF16, M=4, N=16, dy=A, lddy=16, x=B, ldx=16, w=C, stats=D, dx=E_, lddx=16, dw=F_, db=G, ws=WS, bytes=1 << 20):
    return lib.layer_norm_backward(type, M, N, dy, lddy, x, ldx, w, stats, dx, lddx, dw, db, ws, bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=5), -7), (dict(M=-1), -1), (dict(lddy=15), -2), (dict(ldx=15), -2), (dict(lddx=15), -2), (dict(dy=None), -3), (dict(x=None), -3),
    (dict(stats=None), -3), (dict(ws=None), -3), (dict(ws=WS + 16), -7), (dict(bytes=8), -7), (dict(dx=E_ + 1), -7), (dict(dx=A), -4),
    (dict(dw=G), -4), (dict(ws=F_), -4), (dict(dx=D), -4), (dict(dx=None, dw=None, db=None), 0), (dict(N=0, ws=None), 0),
])
def test_norm_backward_refusals(lib, kw, code):
    assert norm_back(lib, **kw) == code


def loss(lib, type=BF16, M=4, N=32, K=16, x=A, ldx=16, w=B, ldw=32, order=0, t=C, tb=8, loss=D, lse=E_, ws=WS, bytes=1 << 20):
    return lib.linear_cross_entropy_forward(type, M, N, K, x, ldx, w, ldw, order, t, tb, loss, lse, ws, bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), -7), (dict(order=2), -7), (dict(tb=2), -7), (dict(M=-1), -1), (dict(N=-1), -1), (dict(K=-1), -1),
    (dict(N=2 ** 31 - 1, ldw=2 ** 31), -1), (dict(ldx=15), -2), (dict(ldw=31), -2), (dict(ldw=15, order=1), -2), (dict(x=None), -3),
    (dict(w=None), -3), (dict(t=None), -3), (dict(loss=None), -3), (dict(lse=None), -3), (dict(ws=None), -3), (dict(x=A + 1), -7),
    (dict(t=C + 4), -7), (dict(loss=D + 2), -7), (dict(ws=WS + 64), -7), (dict(bytes=16), -7), (dict(loss=A), -4), (dict(lse=B), -4),
    (dict(loss=C), -4), (dict(lse=D + 8), -4), (dict(ws=A - 0x100, bytes=1 << 20), -4), (dict(M=0, x=None, w=None, t=None), 0),
])
def test_loss_refusals(lib, kw, code):
    assert loss(lib, **kw) == code


def loss_back(lib, type=BF16, M=4, N=32, K=16, g=C, e=None, x=A, ldx=16, w=B, ldw=32, order=0, t=D, tb=8, lse=E_, dx=F_, lddx=16, dw=G, lddw=32,
              ws=WS, bytes=1 << 20):
    return lib.linear_cross_entropy_backward(type, M, N, K, g, e, x, ldx, w, ldw, order, t, tb, lse, dx, lddx, dw, lddw, ws, bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), -7), (dict(tb=1), -7), (dict(M=-1), -1), (dict(ldx=15), -2), (dict(ldw=31), -2), (dict(lddx=15), -2), (dict(lddw=31), -2),
    (dict(x=None), -3), (dict(w=None), -3), (dict(t=None), -3), (dict(lse=None), -3), (dict(ws=None), -3), (dict(g=C + 2), -7),
    (dict(e=C + 2), -7), (dict(lse=E_ + 1), -7), (dict(dx=F_ + 1), -7), (dict(bytes=16), -7), (dict(ws=WS + 128), -7), (dict(dx=A), -4),
    (dict(dw=B), -4), (dict(dx=G), -4), (dict(dw=E_ - 64), -4), (dict(ws=G), -4), (dict(dx=None, dw=None), 0), (dict(K=0), 0),
])
def test_loss_backward_refusals(lib, kw, code):
    assert loss_back(lib, **kw) == code


def test_workspace_sizes(lib):
    size = lib.layer_norm_backward_workspace_size
    assert size(0, 16, 1, 1) == 0 and size(16, 0, 1, 1) == 0 and size(16, 16, 0, 0) == 0 and size(16, 16, 1, 0) > 0
    assert size(10 ** 6, 4096, 1, 1) < 2 * 152 * 4096 * 4 + 4 * 10 ** 6 + 1024  # the sums of one block an SM, and a number a row
    size = lib.linear_cross_entropy_forward_workspace_size
    assert size(BF16, 0, 32, 16, A, 16, B, 32, 0) == 0 and size(BF16, -1, 32, 16, A, 16, B, 32, 0) == 0
    assert size(BF16, 4, 32, 16, A, 16, B, 32, 0) == 256 + 256                 # two numbers a token and 32 columns; one a token
    assert size(BF16, 4, 32, 16, A + 2, 16, B, 32, 0) == 256 + 256 + 256       # a copy of x
    size = lib.linear_cross_entropy_backward_workspace_size
    assert size(BF16, 4, 32, 16, A, 16, B, 32, 0, 0, 0) == 0 and size(BF16, 4, 32, 0, A, 16, B, 32, 0, 1, 1) == 0
    # at most 2**28 values of dz, whatever the vocabulary, and FP32 sums of dx where it takes several pieces (and
    # several at once where it has few tiles)
    assert size(BF16, 8192, 10 ** 6, 64, A, 64, B, 64, 1, 0, 1) < 2 * 2 ** 28 + 2 ** 20
    assert size(BF16, 8192, 10 ** 6, 512, A, 512, B, 512, 1, 1, 1) - size(BF16, 8192, 10 ** 6, 512, A, 512, B, 512, 1, 0, 1) == 8192 * 512 * 4
    assert size(BF16, 8192, 10 ** 6, 64, A, 64, B, 64, 1, 1, 1) - size(BF16, 8192, 10 ** 6, 64, A, 64, B, 64, 1, 0, 1) == 2 * 8192 * 64 * 4
    assert size(BF16, 1, 1000, 64, A, 64, B, 64, 1, 1, 1) - size(BF16, 1, 1000, 64, A, 64, B, 64, 1, 0, 1) == 64 * 64 * 4


def test_wrappers_refuse_other_tensors(lib):
    torch = pytest.importorskip("torch")
    t, n = torch.ones(4, 4), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: sg.expert_choose(t, 2), lambda: sg.expert_choose_backward(t, t, t.int()), lambda: sg.layer_norm(t),
                 lambda: sg.layer_norm_backward(t, t, None, t), lambda: sg.linear_cross_entropy(t, t, n),
                 lambda: sg.linear_cross_entropy_backward(t[0], t, t, n, t[0])):
        with pytest.raises(TypeError):
            call()


@pytest.fixture(params=["extension", "interpreter"])
def calls(request, lib, monkeypatch, tmp_path):
    """The calls with stand-ins for CUDA tensors, torch and the library's functions; `does` answers them."""
    import ctypes

    import torch

    from dense_fp32_tiled_gb300 import _layers
    from tests import _stand_ins as S
    stand_in = S.install(monkeypatch, lib, request.param, str(tmp_path))
    names = [f for op in ("layer_norm_backward", "linear_cross_entropy_forward", "linear_cross_entropy_backward") for f in (op, op + "_workspace_size")]
    names += ["layer_norm_forward", "expert_choose", "expert_choose_backward"]
    for name in names:
        real = getattr(lib, name)
        back = ctypes.CFUNCTYPE(real.restype, *real.argtypes)(lambda *a, name=name: stand_in.does.get(name, lambda *a: 0)(*a))
        stand_in.callbacks[name] = back
        setattr(stand_in, name, back)
    if request.param == "extension":
        _layers._fast.bind_more({n: ctypes.cast(stand_in.callbacks[n], ctypes.c_void_p).value for n in names}, _layers.SCORINGS)
    return stand_in, S, torch


def test_scratch_is_its_calls_own(calls):
    lib, S, torch = calls
    x, w, t, f = S.Tensor((20, 8)), S.Tensor((8, 16)), S.Tensor((20,), torch.int64), S.Tensor((20,), torch.float32)
    stats = S.Tensor((20, 2), torch.float32)
    for name, call, from_end in (("layer_norm_backward", lambda: sg.layer_norm_backward(x, x, None, stats), 3),
                                 ("linear_cross_entropy_forward", lambda: sg.linear_cross_entropy(x, w, t), 3),
                                 ("linear_cross_entropy_backward", lambda: sg.linear_cross_entropy_backward(f, x, w, t, f), 3)):
        seen, alive = [], []

        def addresses():
            gc.collect()
            return {m().data_ptr() for m in lib.made if m() is not None and m().dtype is torch.uint8}

        def enqueue(*args):
            seen.append(args[-from_end])
            if len(seen) == 1:
                call()
            alive.append(args[-from_end] in addresses())
            return 0

        lib.does[name + "_workspace_size"] = lambda *a: 4096
        lib.does[name] = enqueue
        call()
        assert len(seen) == 2 and seen[0] and seen[1] and seen[0] != seen[1], name
        assert alive == [True, True] and not addresses()


def test_statuses_become_errors(calls):
    lib, S, torch = calls
    x, w, t, f = S.Tensor((20, 8)), S.Tensor((8, 16)), S.Tensor((20,), torch.int64), S.Tensor((20,), torch.float32)
    c, g = S.Tensor((20, 2), torch.int32), S.Tensor((20, 2), torch.float32)
    for name, call in (("layer_norm_forward", lambda: sg.layer_norm(x)), ("layer_norm_backward", lambda: sg.layer_norm_backward(x, x, None, g)),
                       ("expert_choose", lambda: sg.expert_choose(x, 2)), ("expert_choose_backward", lambda: sg.expert_choose_backward(g, x, c)),
                       ("linear_cross_entropy_forward", lambda: sg.linear_cross_entropy(x, w, t)),
                       ("linear_cross_entropy_backward", lambda: sg.linear_cross_entropy_backward(f, x, w, t, f))):
        call()
        lib.does[name] = lambda *a: -5
        with pytest.raises(sg.SgemmError):
            call()


def test_arguments_arrive(calls):
    lib, S, torch = calls
    seen = {}
    for name in ("layer_norm_forward", "expert_choose", "expert_choose_backward", "linear_cross_entropy_forward", "linear_cross_entropy_backward",
                 "layer_norm_backward"):
        lib.does[name] = lambda *a, name=name: seen.__setitem__(name, a) or 0
    x = S.Tensor((20, 8), strides=(12, 1))
    wt, wn, t32 = S.Tensor((16, 8)), S.Tensor((8, 16)), S.Tensor((20,), torch.int32)
    v, f, stats = S.Tensor((8,)), S.Tensor((20,), torch.float32), S.Tensor((20, 2), torch.float32)
    bias = S.Tensor((8,), torch.float32)
    sg.layer_norm(x, v, None, eps=0.25, stats=stats)
    assert seen["layer_norm_forward"][:9] == (1, 20, 8, x.data_ptr(), 12, v.data_ptr(), None, 0.25, stats.data_ptr())
    dx, dw, db = sg.layer_norm_backward(x, x, v, stats, need_dx=False)
    assert dx is None and dw.shape == (8,) and db.shape == (8,) and seen["layer_norm_backward"][9] is None
    chosen, w = sg.expert_choose(x, 3, bias=bias, scoring="sigmoid", groups=4, kept_groups=2, group_top=2, renormalize=False, scale=2.5)
    assert seen["expert_choose"][:13] == (1, 20, 8, 3, x.data_ptr(), 12, bias.data_ptr(), 1, 4, 2, 2, 0, 2.5)
    assert chosen.shape == (20, 3) and chosen.dtype is torch.int32 and w.dtype is torch.float32
    d = sg.expert_choose_backward(w, x, chosen, scoring="sigmoid", renormalize=False, scale=2.5)
    assert seen["expert_choose_backward"][:11] == (1, 20, 8, 3, w.data_ptr(), chosen.data_ptr(), x.data_ptr(), 12, 1, 0, 2.5) and d.shape == (20, 8)
    loss, lse = sg.linear_cross_entropy(x, wt.transpose(0, 1), t32)
    assert seen["linear_cross_entropy_forward"][:11] == (1, 20, 16, 8, x.data_ptr(), 12, wt.data_ptr(), 8, 1, t32.data_ptr(), 4)
    dx, dw = sg.linear_cross_entropy_backward(f, x, wt.transpose(0, 1), t32, lse)
    a = seen["linear_cross_entropy_backward"]
    assert a[4:6] == (f.data_ptr(), None) and a[15] == 8 and a[17] == 8 and dw.shape == (8, 16) and dw.stride() == (1, 8)
    dx, dw = sg.linear_cross_entropy_backward(f, x, wn, t32, lse, dlse=f, need_dx=False)
    a = seen["linear_cross_entropy_backward"]
    assert dx is None and a[5] == f.data_ptr() and a[10] == 0 and a[14] is None and a[17] == 16 and dw.stride() == (16, 1)
