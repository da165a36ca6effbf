"""linear for few tokens: every count around the kernels' limits, features too few
to fill the GPU (K shared out over a cluster), odd sizes and rows, infinities."""
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


def _check(M, N, K, dtype, order, act="silu", pad=0, offset=0):
    g = L.rng(M * 131 + N * 17 + K + order)
    x = L.strided(g, M, K, dtype, pad, offset)
    w = L.weight(g, K, N, dtype, order)
    b, r = L.randn(g, (N,), dtype, 0.5), L.strided(g, M, N, dtype, pad, offset)
    z = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    out = torch.full((M, N + 3), 9.0, dtype=dtype, device="cuda")
    got = sg.linear(x, w, bias=b, residual=r, activation=act, preact=z, out=out[:, :N])
    y, yb, zr, zb = L.forward_ref(x, w, b, r, act)
    L.assert_within(got, y, yb, f"{M}x{N}x{K} {dtype} order {order}")
    L.assert_within(z, zr, zb, f"{M}x{N}x{K} {dtype} order {order} preact")
    assert (out[:, N:] == 9.0).all()


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("order", [0, 1])
@pytest.mark.parametrize("M", [1, 2, 4, 5, 8, 9, 16, 17, 31, 32, 33, 48, 49, 63, 64, 65])
def test_tokens(dtype, order, M):
    _check(M, 72, 328, L.TYPES[dtype], order)
    _check(M, 45, 219, L.TYPES[dtype], order, "gelu", pad=1, offset=1)


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("order", [0, 1])
@pytest.mark.parametrize("size", [(1, 8, 9000), (7, 32, 8192), (12, 200, 4100), (16, 33, 5003), (30, 256, 8192), (17, 2048, 2048), (64, 8, 16384),
                                  (40, 1, 6001), (64, 1000, 1024), (50, 600, 2048), (16, 1100, 1024)],
                         ids=lambda s: "x".join(map(str, s)))
def test_few_features(dtype, order, size):
    _check(*size, L.TYPES[dtype], order)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("order", [0, 1])
@pytest.mark.parametrize("N,K,pad,offset", [(30, 1030, 0, 0), (262, 778, 2, 2), (30, 500, 4, 0), (36, 500, 4, 4), (5000, 98, 2, 0),
                                            (5001, 99, 0, 0), (5004, 100, 0, 0)])
def test_even_and_odd_rows(dtype, order, N, K, pad, offset):
    _check(11, N, K, L.TYPES[dtype], order, pad=pad, offset=offset)


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("M", [3, 12, 40])
def test_infinities_stay_in_their_row_and_column(dtype, M):
    g = L.rng(M)
    dt = L.TYPES[dtype]
    x, w = L.randn(g, (M, 500), dt), L.randn(g, (500, 70), dt)
    x[1, 77], x[2, 499], w[123, 11] = float("inf"), float("nan"), float("-inf")
    got = sg.linear(x, w)
    bad = torch.zeros(M, 70, dtype=torch.bool, device="cuda")
    bad[1], bad[2], bad[:, 11] = True, True, True
    assert torch.equal(~torch.isfinite(got), bad)


@pytest.mark.parametrize("M", [5, 20, 64])
def test_fp32_extremes(M):
    """Largest values, values next to them, and small ones that FP32 still holds whole in three pieces."""
    g = L.rng(M)
    x, w = L.randn(g, (M, 256), torch.float32), L.randn(g, (256, 40), torch.float32)
    x[0] *= 2.0 ** -90
    x[1, :] = 0.0
    x[1, 3], w[3, 5] = 3.4028234663852886e38, 0.5
    w[:, 7] *= 2.0 ** 60
    y = x.double() @ w.double()
    S = x.double().abs() @ w.double().abs()
    got = sg.linear(x, w)
    finite = y.abs() < 3.4e38
    assert torch.isfinite(got[finite]).all()
    L.assert_within(got[finite], y[finite], L.product_bound(256, S, torch.float32)[finite], "extremes")


@pytest.mark.parametrize("dtype", L.TYPES)
def test_same_bits_every_time(dtype):
    g = L.rng(5)
    dt = L.TYPES[dtype]
    for M, N, K in ((16, 96, 4096), (48, 96, 4096)):
        x, w = L.randn(g, (M, K), dt), L.randn(g, (K, N), dt)
        first = sg.linear(x, w)
        assert all(torch.equal(first, sg.linear(x, w)) for _ in range(5))


@pytest.mark.parametrize("dtype", L.TYPES)
def test_in_a_graph(dtype):
    """Clusters and programmatic launches captured and replayed, one product's result the next one's input."""
    g = L.rng(6)
    dt = L.TYPES[dtype]
    for M in (3, 16, 40):
        x = L.randn(g, (M, 4096), dt)
        w1, w2 = L.randn(g, (4096, 96), dt, 1 / 64), L.randn(g, (96, 72), dt, 1 / 8)
        h, y = torch.empty((M, 96), dtype=dt, device="cuda"), torch.empty((M, 72), dtype=dt, device="cuda")
        want = sg.linear(sg.linear(x, w1, activation="relu"), w2)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sg.linear(x, w1, activation="relu", out=h)
            sg.linear(h, w2, out=y)
        for _ in range(3):
            h.zero_(), y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)
