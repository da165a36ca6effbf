"""The gradient of linear_cross_entropy where the vocabulary is taken in several pieces and
dx is the sum of shares of each, side by side (needs a GB300): the shares of all
pieces go into the same sums, which are joined at the end.

Some tokens' dx and some columns of dw against the formulas in 64 bits, with the bounds
of test_cross_entropy_gpu."""
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_tiled_gb300 as sg
from tests import _layers as L
from tests.test_cross_entropy_gpu import U, inputs, reference

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


SIZES = [(6000, 65536, 64), (6000, 90001, 40), (9000, 29697, 128), (2000, 400000, 16)]


def pieces(M, N):
    """Columns of a piece, and of the last one: 2**28 values of M tokens at a time."""
    most = max(1, 2 ** 28 // (-(-M // 8) * 8) // 256) * 256
    n = -(-N // most)
    piece = min(N, -(-(-(-N // n)) // 256) * 256)
    return piece, N - (-(-N // piece) - 1) * piece


def test_sizes_take_several_pieces():
    assert [pieces(M, N) for M, N, _ in SIZES] == [(32768, 32768), (30208, 29585), (15104, 14593), (133376, 133248)]
    # and the tiles of dx are at most half of the SMs, so that its sum is shared out
    assert all(-(-M // 128) * -(-K // 128) <= 76 for M, _, K in SIZES)


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("order", [0, 1])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_shares_of_pieces(dtype, order, M, N, K):
    dt = L.TYPES[dtype]
    g = L.rng(M + N)
    x, w, targets = inputs(g, M, N, K, dt, order, drop=0.05)
    loss, lse = sg.linear_cross_entropy(x, w, targets)
    dloss = torch.rand((M,), generator=g, device="cuda") / M
    dlse = torch.randn((M,), generator=g, device="cuda") * 1e-2 / M
    dx, dw = sg.linear_cross_entropy_backward(dloss, x, w, targets, lse, dlse=dlse)
    only, none = sg.linear_cross_entropy_backward(dloss, x, w, targets, lse, dlse=dlse, need_dw=False)
    assert none is None and torch.equal(only, dx)
    again, _ = sg.linear_cross_entropy_backward(dloss, x, w, targets, lse, dlse=dlse)
    assert torch.equal(again, dx)
    some = (targets >= 0) & (targets < N)
    gd = torch.where(some, dloss.double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    a = gd + dlse.double()
    most = max(float(a.abs().max()), float(gd.abs().max()))
    low = most * 2.0 ** -39 if dtype == "f16" else 0.0

    def dz_of(rows, cols):
        """(dz, a bound of its error) of these tokens and columns."""
        z = x[rows].double() @ w[:, cols].double()
        zb = L.product_bound(K, x[rows].double().abs() @ w[:, cols].double().abs(), dt)
        le = lse[rows].double()[:, None]
        p = torch.exp(z - le) * a[rows][:, None]
        at = torch.arange(N, device="cuda")[cols][None, :] == torch.where(some[rows], targets[rows], torch.full_like(targets[rows], -1))[:, None]
        dz = p - at * gd[rows][:, None]
        e = p.abs() * (zb + 4 * U * (z.abs() + le.abs()) + 2.0 ** -21) + 4 * U * (dz.abs() + at * gd[rows][:, None])
        if dt != torch.float32:
            e = e + L.UNIT[dt] * (dz.abs() + e) + low
        return dz, e

    rows = torch.randint(0, M, (200,), generator=g, device="cuda")
    dz, e = dz_of(rows, slice(0, N))
    wd = w.double()
    ref = dz @ wd.t()
    L.assert_within(dx[rows], ref, e @ wd.abs().t() + L.product_bound(N, (dz.abs() + e) @ wd.abs().t(), dt) + L.rounding(ref, dt), "dx")
    piece, _ = pieces(M, N)
    edges = [c for b in range(0, N + 1, piece) for c in (b - 1, b) if 0 <= c < N] + [N - 1]
    cols = torch.cat([torch.tensor(edges, device="cuda"), torch.randint(0, N, (200,), generator=g, device="cuda")])
    dz, e = dz_of(torch.arange(M, device="cuda"), cols)
    xd = x.double()
    ref = xd.t() @ dz
    L.assert_within(dw[:, cols], ref, xd.abs().t() @ e + L.product_bound(M, xd.abs().t() @ (dz.abs() + e), dt) + L.rounding(ref, dt), "dw")
