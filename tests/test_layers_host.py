"""Refusals of the layer operators, all before any CUDA call (CPU only): the
C ABI's status codes, the workspace sizes, and the Python wrappers' errors."""
import ctypes

import pytest

import dense_fp32_tiled_gb300 as sg
from dense_fp32_tiled_gb300 import build as sg_build

A, B, C, D, E_, F_, WS = (0x10000 * (i + 1) for i in range(7))  # never dereferenced
BF16, F32, F16 = 1, 0, 2


@pytest.fixture(scope="module")
def lib():
    sg_build.build()
    return sg.load_library()


def forward(lib, type=BF16, M=16, N=16, K=16, x=A, ldx=16, w=B, ldw=16, order=0, bias=None, res=None, ldr=0, act=0, z=None,
            ldz=0, y=C, ldy=16, ws=None, bytes=0):
    return lib.linear_forward(type, M, N, K, x, ldx, w, ldw, order, bias, res, ldr, act, z, ldz, y, ldy, ws, bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), -7), (dict(type=-1), -7), (dict(act=5), -7), (dict(act=-1), -7), (dict(order=2), -7),
    (dict(M=-1), -1), (dict(N=-1), -1), (dict(K=-1), -1), (dict(K=2 ** 31 - 1, ldx=2 ** 31, ldw=2 ** 31, order=1), -1),
    (dict(ldx=15), -2), (dict(ldw=15), -2), (dict(ldw=15, order=1), -2), (dict(ldy=15), -2),
    (dict(res=D, ldr=15), -2), (dict(z=D, ldz=15), -2),
    (dict(x=None), -3), (dict(w=None), -3), (dict(y=None), -3),
    (dict(x=A + 2), -3),                                        # needs a copy, and there is no workspace
    (dict(type=F32, M=65), -3),                                 # so do FP32's pieces (more than 64 tokens)
    (dict(x=A + 1, ws=WS, bytes=1 << 20), -7),                  # not aligned to its element
    (dict(y=C + 1), -7), (dict(bias=D + 1), -7),
    (dict(x=A + 2, ws=WS + 128, bytes=1 << 20), -7),            # workspace not 256-byte aligned
    (dict(x=A + 2, ws=WS, bytes=16), -7),                       # too small
    (dict(y=A + 32), -4), (dict(y=B + 64), -4), (dict(z=C + 16, ldz=16), -4), (dict(z=A, ldz=16), -4),
    (dict(res=C + 2, ldr=16), -4), (dict(res=C, ldr=24), -4),   # residual over y, not y itself
    (dict(bias=C + 8), -4), (dict(x=A + 2, ws=C, bytes=1 << 20), -4),
    (dict(M=0), 0), (dict(N=0, ldw=1, ldy=1), 0), (dict(M=0, x=None, w=None, y=None), 0),
])
def test_forward_refusals(lib, kw, code):
    kw = {"M": 17, **kw}
    assert forward(lib, **kw) == code


def backward(lib, type=BF16, M=17, N=16, K=16, dy=A, lddy=16, x=B, ldx=16, w=C, ldw=16, order=0, z=None, ldz=0, act=0, dx=D,
             lddx=16, dw=E_, lddw=16, db=None, ws=None, bytes=0):
    return lib.linear_backward(type, M, N, K, dy, lddy, x, ldx, w, ldw, order, z, ldz, act, dx, lddx, dw, lddw, db, ws, bytes,
                               None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=9), -7), (dict(M=-2), -1), (dict(lddy=15), -2), (dict(ldx=15), -2), (dict(ldw=15), -2), (dict(lddx=15), -2),
    (dict(lddw=15), -2), (dict(act=2), -2), (dict(act=2, ldz=16), -7), (dict(z=F_, ldz=16), -7),
    (dict(dy=None), -3), (dict(x=None), -3), (dict(w=None), -3), (dict(db=F_), -3), (dict(act=2, z=F_, ldz=16), -3),
    (dict(dx=A), -4), (dict(dw=B), -4), (dict(dx=E_), -4), (dict(db=D, ws=WS, bytes=1 << 20), -4),
    (dict(db=F_, ws=D, bytes=1 << 20), -4), (dict(db=F_, ws=WS, bytes=4), -7), (dict(dx=D + 1), -7),
    (dict(dx=None, dw=None), 0),
])
def test_backward_refusals(lib, kw, code):
    assert backward(lib, **kw) == code


def expert(lib, type=BF16, R=20, N=16, K=16, E=3, off=D, x=A, ldx=16, w=B, ldw=16, step=256, order=0, y=C, ldy=16, ws=None, bytes=0):
    return lib.expert_linear_forward(type, R, N, K, E, off, x, ldx, w, ldw, step, order, None, None, 0, 0, None, 0, y, ldy, ws,
                                     bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(E=-1), -1), (dict(E=4097), -1), (dict(off=None), -3), (dict(off=D + 2), -7), (dict(step=255), -2), (dict(step=0), -2),
    (dict(y=D - 600), -4), (dict(y=B + 1024), -4), (dict(x=A + 2), -3), (dict(R=0), 0),
])
def test_expert_refusals(lib, kw, code):
    assert expert(lib, **kw) == code


@pytest.mark.parametrize("fn,args,code", [
    ("expert_sort", (4, 2, 8, A, 3, B, C, None, 0, None), -7),          # choices of 3 bytes
    ("expert_sort", (-1, 2, 8, A, 4, B, C, None, 0, None), -1),
    ("expert_sort", (4, 65, 8, A, 4, B, C, None, 0, None), -1),         # too many choices
    ("expert_sort", (4, 2, 0, A, 4, B, C, None, 0, None), -1),
    ("expert_sort", (4, 2, 4097, A, 4, B, C, None, 0, None), -1),
    ("expert_sort", (4, 2, 8, None, 4, B, C, None, 0, None), -3),
    ("expert_sort", (4, 2, 8, A, 4, B, None, None, 0, None), -3),
    ("expert_sort", (9000, 2, 8, A, 4, B, C, None, 0, None), -3),       # needs a workspace
    ("expert_sort", (9000, 2, 8, A, 4, A + 0x100000, C, WS, 64, None), -7),
    ("expert_sort", (4, 2, 8, A + 4, 8, B, C, None, 0, None), -7),      # 64-bit choices on a 4-byte boundary
    ("expert_sort", (4, 2, 8, A, 4, A + 16, C, None, 0, None), -4),
    ("expert_sort", (4, 2, 8, A, 4, B, B + 8, None, 0, None), -4),
    ("expert_gather", (7, 4, 2, 16, 8, A, B, C, 16, D, 16, None), -7),
    ("expert_gather", (1, 4, 2, -1, 8, A, B, C, 16, D, 16, None), -1),
    ("expert_gather", (1, 4, 2, 16, 8, A, B, C, 15, D, 16, None), -2),
    ("expert_gather", (1, 4, 2, 16, 8, A, B, C, 16, D, 15, None), -2),
    ("expert_gather", (1, 4, 2, 16, 8, None, B, C, 16, D, 16, None), -3),
    ("expert_gather", (1, 4, 2, 16, 8, A, B, C, 16, C + 64, 16, None), -4),
    ("expert_gather", (1, 4, 2, 16, 8, A, B, C + 1, 16, D, 16, None), -7),
    ("expert_gather", (1, 0, 2, 16, 8, None, None, None, 16, None, 16, None), 0),
    ("expert_combine", (1, 4, 2, 16, A, B, C, 15, None, 0, D, 16, None), -2),
    ("expert_combine", (1, 4, 2, 16, A, B, C, 16, E_, 15, D, 16, None), -2),
    ("expert_combine", (1, 4, 2, 16, None, B, C, 16, None, 0, D, 16, None), -3),
    ("expert_combine", (1, 4, 2, 16, A, B, C, 16, D + 2, 16, D, 16, None), -4),
    ("expert_combine", (1, 4, 2, 16, A, B, C, 16, None, 0, C, 16, None), -4),
    ("expert_combine", (1, 4, 2, 16, A, B + 2, C, 16, None, 0, D, 16, None), -7),
    ("expert_combine", (1, 4, 2, 0, None, None, None, 1, None, 0, None, 1, None), 0),
    ("expert_combine_backward", (1, 4, 2, 16, 8, A, B, None, C, 16, D, 15, E_, 16, F_, None), -2),
    ("expert_combine_backward", (1, 4, 2, 16, 8, A, B, None, C, 16, None, 16, E_, 16, F_, None), -3),
    ("expert_combine_backward", (1, 4, 2, 16, 8, A, B, None, C, 16, D, 16, D, 16, F_, None), -4),
    ("expert_combine_backward", (1, 4, 2, 16, 8, A, B, None, C, 16, D, 16, E_, 16, E_ + 64, None), -4),
    ("expert_combine_backward", (1, 4, 2, 16, 8, A, B, None, C, 16, D, 16, E_, 16, F_ + 2, None), -7),
])
def test_route_refusals(lib, fn, args, code):
    assert getattr(lib, fn)(*args) == code


def test_workspace_sizes(lib):
    size = lib.linear_forward_workspace_size
    assert size(BF16, 100, 64, 64, A, 64, B, 64, 0) == 0                       # read as they are
    assert size(BF16, 100, 64, 64, A + 2, 64, B, 64, 0) == 100 * 64 * 2        # a copy of x
    assert size(BF16, 100, 63, 64, A, 64, B, 63, 0) == 64 * 64 * 2             # of w, rows rounded up to 8
    assert size(F32, 100, 64, 64, A, 64, B, 64, 0) == (100 + 64) * 64 * 6      # three pieces of both
    assert size(F32, 16, 64, 64, A, 64, B, 64, 0) == 0                         # few tokens: none
    assert size(BF16, 0, 64, 64, A, 64, B, 64, 0) == 0 and size(BF16, -1, 64, 64, A, 64, B, 64, 0) == 0
    back = lib.linear_backward_workspace_size
    assert back(BF16, 64, 64, 64, A, 64, B, 64, C, 64, 0, 0, 1, 1, 0) == 0     # dz is dy
    assert back(BF16, 64, 64, 64, A, 64, B, 64, C, 64, 0, 2, 1, 1, 0) == 64 * 64 * 2
    assert back(BF16, 64, 64, 64, A, 64, B, 64, C, 64, 0, 0, 0, 0, 1) == (1 + 1) * 64 * 4
    assert lib.expert_sort_workspace_size(8, 2, 16) == 0 and lib.expert_sort_workspace_size(8192, 2, 16) > 0


def test_timeout_query_needs_a_place(lib):
    assert lib.linear_timeouts(ctypes.POINTER(ctypes.c_uint)()) == -3


def test_wrappers_refuse_other_tensors(lib):
    torch = pytest.importorskip("torch")
    t = torch.ones(4, 4)
    for call in (lambda: sg.linear(t, t), lambda: sg.linear_backward(t, t, t), lambda: sg.expert_linear(t, t[None], t),
                 lambda: sg.expert_sort(t, 4), lambda: sg.expert_sort(t.int(), 4), lambda: sg.expert_gather(t, t, t),
                 lambda: sg.expert_combine(t, t), lambda: sg.expert_combine_backward(t, t, t, t, t)):
        with pytest.raises(TypeError):
            call()
