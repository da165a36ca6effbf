"""layer_norm and its gradient against the formulas in 64 bits (needs a GB300).

Bounds, in units u = 2**-24 of FP32.  K bounds the additions that one value goes
through in a row's sum: 64 in a thread (wide rows: N / 512), ten across the
block, some for what is summed.  The sum of the differences has an error of
K u mean|d|, which is left of the mean; the variance, a sum of squares, K + 3 u
of itself, so 1 / deviation (K + 3) / 2 + 2 u.  So h is off by at most
(K + 8) u (|h| + 2).  In dx = rstd (g - mean g - h mean(g h)) the means are off
by K u of the means of the magnitudes G and GH, and by h's error times G.  A
column's sum goes through M / 304 additions in a block, 16 across its warps and
42 over the blocks.
"""
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_tiled_gb300 as sg
from tests import _layers as L

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_fp32_tiled_gb300 import build
    build.build()
    sg.load_library()


def adds(N):
    return 80 + N / 512


def h_of(x, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + eps)
    return (x - mean) * rstd, mean, rstd


def check_forward(x, weight, bias, eps, out=None):
    M, N = x.shape
    stats = torch.full((M, 2), float("nan"), device="cuda")
    y = sg.layer_norm(x, weight, bias, eps=eps, stats=stats, out=out)
    h, mean, rstd = h_of(x, eps)
    w = weight.double() if weight is not None else torch.ones(N, dtype=torch.float64, device="cuda")
    b = bias.double() if bias is not None else torch.zeros(N, dtype=torch.float64, device="cuda")
    ref = h * w + b
    K = adds(N)
    bound = (K + 8) * U * (h.abs() + 2) * w.abs() + 2 * U * (ref.abs() + (h * w).abs()) + L.rounding(ref, x.dtype)
    L.assert_within(y, ref, bound, "y")
    d = (x.double() - mean).abs().mean(1, keepdim=True)
    L.assert_within(stats[:, :1], mean, 2 * U * mean.abs() + (K + 2) * U * d + 1e-30, "mean")
    L.assert_within(stats[:, 1:], rstd, (K / 2 + 5) * U * rstd, "rstd")
    return y, stats


def check_backward(x, dy, weight, eps=1e-5):
    M, N = x.shape
    stats = torch.empty((M, 2), device="cuda")
    sg.layer_norm(x, weight, None, eps=eps, stats=stats)
    dx, dw, db = sg.layer_norm_backward(dy, x, weight, stats)
    h, mean, rstd = h_of(x, eps)
    g = dy.double() * (weight.double() if weight is not None else 1.0)
    ref = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    K = adds(N)
    G, GH = g.abs().mean(1, keepdim=True), (g * h).abs().mean(1, keepdim=True)
    bound = rstd * U * (K + 16) * (g.abs() + 2 * G + 3 * (h.abs() + 2) * (GH + G)) + L.rounding(ref, x.dtype)
    L.assert_within(dx, ref, bound, "dx")
    chain = M / 304 + 80
    hb = (K + 8) * U * (h.abs() + 2)
    ref = (dy.double() * h).sum(0)
    L.assert_within(dw, ref, chain * U * (dy.double() * h).abs().sum(0) + (dy.double().abs() * hb).sum(0) + L.rounding(ref, x.dtype), "dweight")
    ref = dy.double().sum(0)
    L.assert_within(db, ref, chain * U * dy.double().abs().sum(0) + L.rounding(ref, x.dtype), "dbias")
    return dx, dw, db, stats


SHAPES = [(1, 1), (1, 4096), (2, 2), (3, 7), (5, 31), (9, 64), (33, 100), (700, 512), (65, 513), (40, 1000), (21, 1024),
          (6, 1025), (400, 2048), (30, 4095), (12, 4096), (5, 8192), (4, 8193), (3, 16384), (2, 16385), (3, 32768), (2, 33000),
          (1, 70001)]


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("M,N", SHAPES)
def test_forward(dtype, M, N):
    dt = L.TYPES[dtype]
    g = L.rng(M + N)
    for pad, offset in ((0, 0), (8, 0), (3, 1)):
        x = L.strided(g, M, N, dt, pad, offset, scale=2.0)
        weight, bias = L.randn(g, (N,), dt), L.randn(g, (N,), dt)
        out = L.strided(g, M, N, dt, 16 if pad == 8 else pad)
        y, _ = check_forward(x, weight, bias, 1e-5, out=out)
        assert y is out
    check_forward(x, None, None, 0.5)
    check_forward(x, weight, None, 1e-5)
    check_forward(x, None, bias, 1e-5)


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("M,N", SHAPES + [(3000, 64), (2500, 520), (1300, 3000)])
def test_backward(dtype, M, N):
    dt = L.TYPES[dtype]
    g = L.rng(M + N + 1)
    for pad, offset in ((0, 0), (8, 0), (3, 1)):
        x, dy = L.strided(g, M, N, dt, pad, offset, scale=2.0), L.strided(g, M, N, dt, pad)
        check_backward(x, dy, L.randn(g, (N,), dt))
    check_backward(x, dy, None)


@pytest.mark.parametrize("N", [33, 1000, 4096, 9001, 40000])
def test_rows_far_from_zero(N):
    # a mean of 1e4 deviations: what rounding leaves of it would be 6e-4 of a deviation
    g = L.rng(N)
    x = torch.randn((20, N), generator=g, device="cuda") + 1e4
    check_forward(x, None, None, 1e-5)
    check_backward(x, torch.randn((20, N), generator=g, device="cuda"), L.randn(g, (N,), torch.float32))


def test_constant_rows_and_values_out_of_range():
    x = torch.full((3, 300), 7.25, device="cuda")
    stats = torch.empty((3, 2), device="cuda")
    y = sg.layer_norm(x, None, None, eps=1e-5, stats=stats)
    assert (y == 0).all() and (stats[:, 0] == 7.25).all()
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    y = sg.layer_norm(x)
    assert (y[0] == 0).all() and torch.isnan(y[1]).all() and torch.isnan(y[2, 7])
    # a row's NaN stays in its row, and in its columns' sums
    dx, dw, db = sg.layer_norm_backward(torch.ones_like(x), x, None, torch.tensor([[7.25, 300.0], [7.25, 1.0], [7.25, 1.0]], device="cuda"))
    assert torch.isfinite(dx[0]).all() and torch.isnan(dx[1]).any() and torch.isfinite(db).all()


def test_gradient_against_differences():
    g = L.rng(6)
    x, dy, w = (torch.randn(s, generator=g, device="cuda") for s in ((3, 17), (3, 17), (17,)))
    dx, dw, db, _ = check_backward(x, dy, w)
    step = 1e-5
    f = lambda a, b, c: (dy.double() * (h_of(a, 1e-5)[0] * b + c)).sum()
    a, b, c = x.double(), w.double(), torch.zeros(17, dtype=torch.float64, device="cuda")
    for i in range(17):
        e = torch.zeros(17, dtype=torch.float64, device="cuda")
        e[i] = step
        for r in range(3):
            m = torch.zeros((3, 17), dtype=torch.float64, device="cuda")
            m[r, i] = step
            assert abs((f(a + m, b, c) - f(a - m, b, c)) / (2 * step) - dx[r, i]) < 1e-5
        assert abs((f(a, b + e, c) - f(a, b - e, c)) / (2 * step) - dw[i]) < 1e-5
        assert abs((f(a, b, c + e) - f(a, b, c - e)) / (2 * step) - db[i]) < 1e-5


@pytest.mark.parametrize("N", [500, 4096, 20000])
def test_what_is_not_needed(N):
    g = L.rng(N)
    x, dy, w = L.randn(g, (50, N), torch.bfloat16), L.randn(g, (50, N), torch.bfloat16), L.randn(g, (N,), torch.bfloat16)
    dx, dw, db, stats = check_backward(x, dy, w)
    for need in range(8):
        got = sg.layer_norm_backward(dy, x, w, stats, need_dx=bool(need & 1), need_dweight=bool(need & 2), need_dbias=bool(need & 4))
        for bit, a, b in zip((1, 2, 4), got, (dx, dw, db)):
            assert (a is None) if not need & bit else torch.equal(a, b)
    assert torch.equal(sg.layer_norm(x, w, w), sg.layer_norm(x, w, w, stats=torch.empty((50, 2), device="cuda")))


def test_empty_and_refused():
    x, w = torch.ones((4, 8), device="cuda"), torch.ones(8, device="cuda")
    stats = torch.full((4, 2), 5.0, device="cuda")
    assert sg.layer_norm(x[:0], w).shape == (0, 8)
    assert sg.layer_norm(x[:, :0], stats=stats).shape == (4, 0) and (stats == 0).all()
    dx, dw, db = sg.layer_norm_backward(x[:0], x[:0], w, stats[:0])
    assert dx.shape == (0, 8) and (dw == 0).all() and (db == 0).all()
    dx, dw, db = sg.layer_norm_backward(x[:, :0], x[:, :0], w[:0], stats)
    assert dx.shape == (4, 0) and dw.shape == (0,)
    for call, error in [(lambda: sg.layer_norm(x[0]), ValueError), (lambda: sg.layer_norm(x.double()), TypeError),
                        (lambda: sg.layer_norm(x.cpu()), TypeError), (lambda: sg.layer_norm(x, w[:7]), ValueError),
                        (lambda: sg.layer_norm(x, w.half()), TypeError), (lambda: sg.layer_norm(x, w, torch.ones(16, device="cuda")[::2]), ValueError),
                        (lambda: sg.layer_norm(x, stats=stats[:3]), ValueError), (lambda: sg.layer_norm(x, stats=stats.half()), TypeError),
                        (lambda: sg.layer_norm(x, eps=-1.0), sg.SgemmError), (lambda: sg.layer_norm(x, eps=float("nan")), sg.SgemmError),
                        (lambda: sg.layer_norm(x, out=x), sg.SgemmError), (lambda: sg.layer_norm(x.t()), ValueError),
                        (lambda: sg.layer_norm_backward(x, x, w, None), ValueError), (lambda: sg.layer_norm_backward(x[:3], x, w, stats), ValueError),
                        (lambda: sg.layer_norm_backward(x.half(), x, w, stats), TypeError)]:
        with pytest.raises(error):
            call()


# Where the blocks' forms change: rows of a warp, several rows a block (their number by the
# rows there are, not a multiple of them), one, two blocks an SM, rows read more than once.
@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("M,N", [(1, 129), (153, 257), (2000, 1001), (1999, 1000), (700, 4097), (611, 4098), (305, 6145), (304, 6148), (153, 8193),
                                 (160, 12288), (155, 12289), (154, 12290), (153, 12296), (5, 14336), (3, 16384), (4, 16386), (3, 24576), (2, 24577)])
@pytest.mark.parametrize("weights", ["both", "weight", "bias", "none"])
def test_forward_forms(dtype, M, N, weights):
    dt = L.TYPES[dtype]
    g = L.rng(M * 7 + N)
    x = L.strided(g, M, N, dt, 0, 0, scale=2.0)
    weight = L.randn(g, (N,), dt) if weights in ("both", "weight") else None
    bias = L.randn(g, (N,), dt) if weights in ("both", "bias") else None
    check_forward(x, weight, bias, 1e-5)


# The gradient's: several rows a block, one, weights in shared memory, in registers, from L1
# (wide rows in FP32), rows read more than once.
@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("M,N", [(1, 129), (153, 257), (2000, 1001), (700, 4097), (611, 4098), (609, 4100), (155, 6145), (160, 7600), (155, 8200),
                                 (154, 8194), (153, 8193), (160, 12288), (155, 12290), (153, 12296), (5, 16384), (4, 16386)])
@pytest.mark.parametrize("weight", [True, False])
def test_backward_forms(dtype, M, N, weight):
    dt = L.TYPES[dtype]
    g = L.rng(M * 5 + N)
    x, dy = L.strided(g, M, N, dt, 0, 0, scale=2.0), L.strided(g, M, N, dt, 0)
    check_backward(x, dy, L.randn(g, (N,), dt) if weight else None)


# Of rows read in pieces: more rows than the column sums' blocks, and fewer.
@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("M,N", [(300, 12289), (1100, 12290), (257, 16388), (33, 24579), (700, 9001), (155, 11999)])
def test_backward_wide(dtype, M, N):
    dt = L.TYPES[dtype]
    g = L.rng(M + 3 * N)
    check_backward(L.strided(g, M, N, dt, 0, 0, scale=2.0), L.strided(g, M, N, dt, 0), L.randn(g, (N,), dt))
