"""FP32 products hold FP32's precision: what the bounds that grow with K cannot
show.  Single products, sums whose leading pieces cancel, and the error's root
mean square, for every number of tokens that has a kernel of its own, every
plan, both gradients and the experts (needs a GB300).

Tolerances.  A single product is off by the products of pieces that are left
out, at most 1.5 * 2**-24 of it with pieces rounded to nearest (|b| <= 2**-8,
|c| <= 2**-17 of the value's binade: b c' + c b' = 2**-24, what a third piece
leaves, 2**-26 each, the same again at most by half), and by the last addition,
which cuts at most a unit in the last place, 2**-23; 5 * 2**-24 allows one
more bit lost in aligning the addends.  Sums of normal numbers: each of a
128-K block's 48 additions cuts half a unit of the running sum on average,
which is 2/3 of the block's in the mean: 48 * 0.5 * 0.72 * 2**-23 * 2/3 =
2**-19.5 of the result; FP32 sums of blocks and the pieces add little.
Cancelling sums: the largest addends are below 2, so an addition cuts at most
2**-22 of what is below them; 2**-20 in all.
"""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

torch = pytest.importorskip("torch")

import dense_fp32_tiled_gb300 as sg
from tests import _layers as L
from tests.test_linear_plans_gpu import PLANS

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOKENS = [1, 4, 5, 16, 17, 40, 64, 65, 300]  # each kernel's first or last, and the product kernel's


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_fp32_tiled_gb300 import build
    build.build()
    sg.load_library()


def _held(w, order):
    """w with either of its dimensions contiguous in memory."""
    return w.transpose(-1, -2).contiguous().transpose(-1, -2) if order else w.contiguous()


def _forward(a, b, order):
    return sg.linear(a, _held(b, order))


def _dx(a, b, order):  # a is dy, b is w's transpose
    w = _held(b.t(), order)
    return sg.linear_backward(a, torch.zeros(a.shape[0], w.shape[0], device="cuda"), w, need_dw=False, need_dbias=False)[0]


def _dw(a, b, order):  # a is x's transpose, b is dy
    x = a.t().contiguous()
    return sg.linear_backward(b, x, _held(torch.zeros(x.shape[1], b.shape[1], device="cuda"), order), need_dx=False, need_dbias=False)[1]


def _experts(a, b, order):
    """All rows with the second of three experts."""
    off = torch.tensor([0, 0, a.shape[0], a.shape[0]], dtype=torch.int32, device="cuda")
    return sg.expert_linear(a, _held(torch.stack([torch.full_like(b, 9.0), b, torch.full_like(b, 9.0)]), order), off)


def _experts_dw(a, b, order):
    """The rows between those of two other experts, whose last tiles hold them too."""
    x, dy = a.t(), b
    x = torch.cat([torch.full((5, x.shape[1]), 9.0, device="cuda"), x, torch.full((7, x.shape[1]), 9.0, device="cuda")])
    dy = torch.cat([torch.full((5, dy.shape[1]), 9.0, device="cuda"), dy, torch.full((7, dy.shape[1]), 9.0, device="cuda")])
    n = b.shape[0]
    off = torch.tensor([0, 5, 5 + n, 12 + n], dtype=torch.int32, device="cuda")
    w = _held(torch.zeros(3, x.shape[1], dy.shape[1], device="cuda"), order)
    return sg.expert_linear_backward(dy, x, w, off, need_dx=False, need_dbias=False)[1][1]


PRODUCTS = {"forward": _forward, "dx": _dx, "dw": _dw, "experts": _experts, "experts dw": _experts_dw}


def _values(g, n):
    """Values in [1, 2) with random low bits; every third has its eight leading bits 1.0000000 and
    the next ones set, where pieces that were cut off rather than rounded would be off the most."""
    v = torch.randint(0, 2 ** 23, (n,), generator=g, device="cuda")
    v[::3] = (v[::3] & 0xff) | 0xff00
    v[0] = 0xffff
    return 1 + v.float() * 2.0 ** -23


def check_single(product, rows, depth, cols, order):
    g = L.rng(rows * 7 + depth + cols)
    a, b = torch.zeros(rows, depth, device="cuda"), torch.zeros(depth, cols, device="cuda")
    at = depth * 2 // 3
    a[:, at], b[at] = _values(g, rows), _values(g, cols)
    want = torch.outer(a[:, at].double(), b[at].double())
    L.assert_within(PRODUCTS[product](a, b, order), want, 5 * 2.0 ** -24 * want, f"{product} {rows}x{cols}x{depth} order {order}")


def check_cancelling(product, rows, depth, cols, order):
    """Columns 0, 3, ..: the third piece of a by the first of b; 1, 4, ..: the first by the third;
    2, 5, ..: the second by the second; everything larger cancels."""
    c, s, t = 3 * 2.0 ** -19, 1 + 2.0 ** -9, 3 * 2.0 ** -10
    scale = 2.0 ** (torch.arange(rows, device="cuda") % 5 - 2)
    a, b = torch.zeros(rows, depth, device="cuda"), torch.zeros(depth, cols, device="cuda")
    want = torch.empty(cols, dtype=torch.float64, device="cuda")
    k = [2 * (depth * i // 8) for i in (0, 2, 3)]  # even: a pair is never parted
    for i, (left, right, value) in enumerate((((s + c, s), (1.0, -1.0), c), ((1.0, -1.0), (s + c, s), c),
                                              ((1 + t, 1.0), (1 + t, -(1 + 2 * t)), t * t))):
        for j in range(2):
            a[:, k[i] + j], b[k[i] + j, i::3] = left[j] * scale, right[j]
        want[i::3] = value
    want = scale.double()[:, None] * want
    assert torch.equal(a.double() @ b.double(), want)
    L.assert_within(PRODUCTS[product](a, b, order), want, 2.0 ** -20 * scale.double()[:, None].expand_as(want),
                    f"{product} {rows}x{cols}x{depth} order {order}")


def check_mean_square(product, rows, depth, cols, order):
    g = L.rng(rows + depth * 3 + cols)
    a, b = L.randn(g, (rows, depth), torch.float32), L.randn(g, (depth, cols), torch.float32)
    want = a.double() @ b.double()
    off = float((PRODUCTS[product](a, b, order).double() - want).norm() / want.norm())
    assert off <= 2.0 ** -19, (product, rows, depth, cols, order, off)


@pytest.mark.parametrize("check", [check_single, check_cancelling, check_mean_square])
@pytest.mark.parametrize("order", [0, 1])
def test_tokens(check, order):
    for rows in TOKENS:
        for depth, cols in ((200, 90), (4096, 33), (331, 61)):
            check("forward", rows, depth, cols, order)


@pytest.mark.parametrize("check", [check_single, check_cancelling, check_mean_square])
@pytest.mark.parametrize("product", list(PRODUCTS)[1:])
def test_gradients_and_experts(check, product):
    for rows, depth, cols in ((7, 200, 90), (150, 331, 200), (90, 2100, 61)):
        for order in (0, 1):
            check(product, rows, depth, cols, order)


def check_plan():
    for check in (check_single, check_cancelling, check_mean_square):
        for product in PRODUCTS:
            check(product, 300, 333, 200, 1)
    assert sg.linear_timeouts() == 0


def test_plans():
    """Every plan, each in a child process (LINEAR_TUNE is read once)."""
    code = "import sys; sys.path.insert(0, %r); from tests.test_fp32_pieces_gpu import check_plan; check_plan()" % ROOT

    def run(plan):
        return plan, subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=dict(os.environ, LINEAR_TUNE=plan),
                                    capture_output=True, text=True, timeout=300)

    with ThreadPoolExecutor(4) as pool:
        for plan, r in pool.map(run, [p for p in PLANS if "bt=256" not in p]):  # 256 wide is for 16 bits
            assert r.returncode == 0, plan + r.stdout[-1000:] + r.stderr[-3000:]


# ---- the ends of FP32's range in the product kernel (65 tokens and more) -------------
@pytest.mark.parametrize("order", [0, 1])
def test_infinities_in_the_product_kernel(order):
    """Each makes every element that it enters NaN or infinite, and no other, whatever it meets."""
    g = L.rng(3)
    for M, N, K in ((70, 70, 500), (200, 130, 4096)):
        x, w = L.randn(g, (M, K), torch.float32), L.randn(g, (K, N), torch.float32)
        w[77, 5] = 0.0
        x[1, 77], x[2, K - 1], w[123, 11] = float("inf"), float("nan"), float("-inf")
        bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
        bad[1], bad[2], bad[:, 11] = True, True, True
        assert torch.equal(~torch.isfinite(sg.linear(x, _held(w, order))), bad)
        dy = L.randn(g, (M, N), torch.float32)
        dy[3, 7] = float("inf")
        dx, dw, db = sg.linear_backward(dy, x, _held(w, order))
        assert not torch.isfinite(dx[3]).any() and not torch.isfinite(dx[:, 123]).any()
        keep_r, keep_k = [i for i in range(M) if i != 3], [k for k in range(K) if k != 123]
        assert torch.isfinite(dx[keep_r][:, keep_k]).all()
        assert not torch.isfinite(dw[:, 7]).any() and not torch.isfinite(dw[77]).any() and not torch.isfinite(dw[K - 1]).any()
        keep_n, keep_k = [n for n in range(N) if n != 7], [k for k in range(K) if k not in (77, K - 1)]
        assert torch.isfinite(dw[keep_k][:, keep_n]).all()
        assert not torch.isfinite(db[7]) and torch.isfinite(db[keep_n]).all()


@pytest.mark.parametrize("order", [0, 1])
def test_extremes_in_the_product_kernel(order):
    """Values whose leading piece would round up to infinity, and small ones that three pieces still hold whole."""
    M, N, K = 70, 40, 256
    g = L.rng(4)
    x, w = L.randn(g, (M, K), torch.float32), L.randn(g, (K, N), torch.float32)
    x[0] *= 2.0 ** -90
    x[1:5] = 0.0
    x[1, 3], x[2, 3], x[3, 3], x[4, 3] = 3.4028234663852886e38, -3.4028234663852886e38, 3.3961775292304957e38, 3.3e38
    w[3, 5] = 0.5
    w[:, 7] *= 2.0 ** 60
    y, S = x.double() @ w.double(), x.double().abs() @ w.double().abs()
    got, finite = sg.linear(x, _held(w, order)), y.abs() < 3.4e38
    assert torch.isfinite(got[finite]).all()
    L.assert_within(got[finite], y[finite], L.product_bound(K, S, torch.float32)[finite], "extremes")
