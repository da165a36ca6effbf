"""linear and linear_backward against the formulas in 64 bits (needs a GB300)."""
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_tiled_gb300 as sg
from tests import _layers as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_fp32_tiled_gb300 import build
    build.build()
    sg.load_library()
    yield
    assert sg.linear_timeouts() == 0


SIZES = [(1, 1, 1), (1, 128, 64), (3, 5, 7), (16, 16, 16), (17, 33, 65), (64, 192, 128), (129, 257, 127),
         (300, 262, 190), (1, 1000, 2049), (5, 640, 4096), (40, 96, 1024), (1000, 1030, 777), (257, 2304, 320)]


def _check_forward(g, M, N, K, dtype, act, order, bias, residual, save, pad=0, offset=0):
    x = L.strided(g, M, K, dtype, pad, offset)
    w = L.weight(g, K, N, dtype, order)
    b = L.randn(g, (N,), dtype, 0.5) if bias else None
    r = L.strided(g, M, N, dtype, pad, offset) if residual else None
    z = torch.full((M, N + pad), 7.0, dtype=dtype, device="cuda") if save else None
    out = torch.full((M, N + pad), 9.0, dtype=dtype, device="cuda")
    got = sg.linear(x, w, bias=b, residual=r, activation=act, preact=z[:, :N] if save else None, out=out[:, :N])
    y, yb, zr, zb = L.forward_ref(x, w, b, r, act)
    what = f"{M}x{N}x{K} {dtype} {act} order {order}"
    L.assert_within(got, y, yb, what)
    if save:
        L.assert_within(z[:, :N], zr, zb, what + " preact")
    if pad:  # nothing past the rows is touched
        assert (out[:, N:] == 9.0).all() and (not save or (z[:, N:] == 7.0).all())


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_forward_sizes(dtype, size):
    M, N, K = size
    g = L.rng(M * 7 + N * 3 + K)
    _check_forward(g, M, N, K, L.TYPES[dtype], L.ACTS[(M + N) % 5], (M + K) % 2, True, True, True)
    _check_forward(g, M, N, K, L.TYPES[dtype], "none", (M + K + 1) % 2, False, False, False)


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("act", L.ACTS)
@pytest.mark.parametrize("order", [0, 1])
def test_forward_activations_and_strides(dtype, act, order):
    g = L.rng(order)
    for pad, offset in ((0, 0), (8, 8), (3, 1), (1, 0)):
        _check_forward(g, 70, 130, 96, L.TYPES[dtype], act, order, True, True, True, pad, offset)


@pytest.mark.parametrize("dtype", L.TYPES)
def test_forward_without_reduction_and_empty(dtype):
    dt = L.TYPES[dtype]
    g = L.rng(1)
    b, r = L.randn(g, (40,), dt), L.randn(g, (6, 40), dt)
    y = sg.linear(torch.empty(6, 0, dtype=dt, device="cuda"), torch.empty(0, 40, dtype=dt, device="cuda"), b, r, "relu")
    want = torch.relu(b.double()) + r.double()
    L.assert_within(y, want, L.rounding(want, dt) + 2.0 ** -22, "K = 0")
    assert sg.linear(torch.empty(0, 5, dtype=dt, device="cuda"), torch.ones(5, 8, dtype=dt, device="cuda")).shape == (0, 8)
    assert sg.linear(torch.ones(4, 5, dtype=dt, device="cuda"), torch.empty(5, 0, dtype=dt, device="cuda")).shape == (4, 0)


@pytest.mark.parametrize("dtype", L.TYPES)
def test_forward_residual_in_place_and_another_stream(dtype):
    dt = L.TYPES[dtype]
    g = L.rng(5)
    x, w = L.randn(g, (33, 100), dt), L.weight(g, 100, 72, dt, 0)
    r = L.randn(g, (33, 72), dt)
    y, yb, _, _ = L.forward_ref(x, w, None, r, "silu")
    acc = r.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = sg.linear(x, w, residual=acc, activation="silu", out=acc, stream=s)
    s.synchronize()
    assert got is acc
    L.assert_within(acc, y, yb, "in place")


@pytest.mark.parametrize("dtype", L.TYPES)
def test_forward_infinities_and_nans(dtype):
    # a NaN or infinity reaches its own row (of x) or column (of w) and nothing else
    dt = L.TYPES[dtype]
    g = L.rng(6)
    x, w = L.randn(g, (50, 130), dt), L.weight(g, 130, 70, dt, 1)
    clean = sg.linear(x, w)
    x2, w2 = x.clone(), w.clone()
    x2[7, 129] = float("nan")
    w2[3, 11] = float("inf")
    got = sg.linear(x2, w2)
    assert torch.isnan(got[7]).all()
    assert not torch.isfinite(got[:, 11]).any()
    keep_r = [i for i in range(50) if i != 7]
    keep_c = [i for i in range(70) if i != 11]
    assert torch.equal(got[keep_r][:, keep_c], clean[keep_r][:, keep_c])


def test_forward_f32_extremes():
    # values whose leading piece would round up to infinity, and tiny ones
    big = torch.tensor([[3.4028235e38, -3.4e38, 1e-30, 1e-38]], device="cuda").repeat(3, 1)
    w = torch.tensor([[0.25, 0.5], [0.125, -0.25], [1e30, 1.0], [0.0, 1e38]], device="cuda")
    want = big.double() @ w.double()
    S = big.double().abs() @ w.double().abs()
    L.assert_within(sg.linear(big, w), want, L.product_bound(4, S, torch.float32), "extremes")


@pytest.mark.parametrize("dtype", L.TYPES)
def test_forward_same_bits_twice(dtype):
    dt = L.TYPES[dtype]
    g = L.rng(8)
    for M, N, K in ((3, 256, 4096), (700, 900, 500)):
        x, w = L.randn(g, (M, K), dt), L.weight(g, K, N, dt, 1)
        assert torch.equal(sg.linear(x, w, activation="gelu"), sg.linear(x, w, activation="gelu"))


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("order", [0, 1])
def test_backward_sizes(dtype, size, order):
    M, N, K = size
    dt = L.TYPES[dtype]
    g = L.rng(M + N * 5 + K * 3)
    for act, pad in ((L.ACTS[(M + N + K) % 5], 0), ("none", 3), ("silu", 8)):
        x, dy = L.strided(g, M, K, dt, pad), L.strided(g, M, N, dt, pad, scale=0.5)
        w = L.weight(g, K, N, dt, order)
        z = L.strided(g, M, N, dt, pad) if act != "none" else None
        got = sg.linear_backward(dy, x, w, preact=z, activation=act)
        for name, t, (ref, bound) in zip(("dx", "dw", "dbias"), got, L.backward_ref(dy, x, w, z, act)):
            L.assert_within(t, ref, bound, f"{name} {M}x{N}x{K} {dtype} {act} pad {pad}")
        assert got[1].stride() == ((1, K) if order and N > 1 and K > 1 else got[1].stride())


@pytest.mark.parametrize("dtype", L.TYPES)
def test_backward_empty_sums(dtype):
    dt = L.TYPES[dtype]
    dx, dw, db = sg.linear_backward(torch.empty(0, 9, dtype=dt, device="cuda"), torch.empty(0, 20, dtype=dt, device="cuda"),
                                    torch.ones(20, 9, dtype=dt, device="cuda"))
    assert dx.shape == (0, 20) and (dw == 0).all() and (db == 0).all()
    dx, dw, db = sg.linear_backward(torch.empty(4, 0, dtype=dt, device="cuda"), torch.ones(4, 20, dtype=dt, device="cuda"),
                                    torch.empty(20, 0, dtype=dt, device="cuda"))
    assert dx.shape == (4, 20) and (dx == 0).all() and dw.shape == (20, 0) and db.shape == (0,)
    dy = torch.ones(3, 5, dtype=dt, device="cuda")
    dx, dw, db = sg.linear_backward(dy, torch.empty(3, 0, dtype=dt, device="cuda"), torch.empty(0, 5, dtype=dt, device="cuda"))
    assert dx.shape == (3, 0) and dw.shape == (0, 5) and (db == 3).all()


def test_backward_only_what_is_needed():
    g = L.rng(9)
    x, dy, w = L.randn(g, (30, 40), torch.float32), L.randn(g, (30, 50), torch.float32), L.weight(g, 40, 50, torch.float32, 0)
    full = sg.linear_backward(dy, x, w)
    for i, keep in enumerate(("need_dx", "need_dw", "need_dbias")):
        flags = {k: k == keep for k in ("need_dx", "need_dw", "need_dbias")}
        got = sg.linear_backward(dy, x, w, **flags)
        for j in range(3):
            assert (got[j] is None) == (i != j)
        assert torch.equal(got[i], full[i])


@pytest.mark.parametrize("act", L.ACTS)
def test_backward_against_differences(act):
    """d(sum dy * y) / d(x, w, b) by central differences of linear's own FP32 result."""
    g = L.rng(10)
    M, N, K = 6, 9, 11
    x, w, b = L.randn(g, (M, K), torch.float32), L.weight(g, K, N, torch.float32, 0), L.randn(g, (N,), torch.float32)
    dy = L.randn(g, (M, N), torch.float32)
    z = torch.empty(M, N, device="cuda")
    sg.linear(x, w, b, activation=act, preact=z)
    if act == "relu":
        assert (z.abs() > 0.02).sum() > 0.9 * z.numel()
    grads = sg.linear_backward(dy, x, w, preact=z if act != "none" else None, activation=act)
    h = 2.0 ** -7

    def loss(x_, w_, b_):
        return (sg.linear(x_, w_, b_, activation=act).double() * dy.double()).sum()

    for t, grad, which in ((x, grads[0], 0), (w, grads[1], 1), (b, grads[2], 2)):
        flat = t.reshape(-1)
        for i in range(0, flat.numel(), 5):
            args = [[x, w, b], [x, w, b]]
            for side, sign in ((0, 1), (1, -1)):
                moved = flat.clone()
                moved[i] += sign * h
                args[side][which] = moved.view_as(t)
            near = z.abs().min()
            if act == "relu" and near < 4 * h:  # a kink inside the step: no derivative to compare with
                zs = [x @ w + b for x, w, b in args]
                if ((zs[0] > 0) != (zs[1] > 0)).any():
                    continue
            # truncation h^2/6 times third derivatives of at most 2 over the terms, rounding 2^-22 over 2 h
            scale = float(dy.abs().sum()) * (1 + float(x.abs().max()) ** 3 + float(w.abs().max()) ** 3)
            diff = (loss(*args[0]) - loss(*args[1])) / (2 * h)
            assert abs(float(diff) - float(grad.reshape(-1)[i])) <= scale * (h * h + 2.0 ** -20 / h), (act, which, i)


def test_graph_capture():
    g = L.rng(11)
    x, w, b = L.randn(g, (64, 256), torch.bfloat16), L.weight(g, 256, 384, torch.bfloat16, 1), L.randn(g, (384,), torch.bfloat16)
    out = torch.empty(64, 384, dtype=torch.bfloat16, device="cuda")
    sg.linear(x, w, b, activation="silu", out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sg.linear(x, w, b, activation="silu", out=out)
    x.copy_(L.randn(g, (64, 256), torch.bfloat16))
    graph.replay()
    assert torch.equal(out, sg.linear(x, w, b, activation="silu"))
