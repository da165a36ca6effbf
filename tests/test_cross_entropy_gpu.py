"""linear_cross_entropy and its gradient against the formulas in 64 bits (needs a GB300).

Bounds, u = 2**-24.  A logit is a product of K terms, within
L.product_bound(K, S) of the true one, S = sum |x||w|; the log sum of
exponentials moves by no more than its largest, zb.  The exponentials are off by
2**-21 (the fast one, and the rounding of its argument for what matters of the
sum), the sum of positive terms by its additions: 16 at a time in a tile, 8 + N /
512 over the tiles' parts, both counted double; the logarithm and the largest
value by their own size.
p = exp(z - lse) is off by zb and the rounding of the exponent, (|z| + |lse|) u.
dz, a fraction of the largest |dloss| and |dloss + dlse|, is rounded to the
16-bit types (float16: times 2**14, so nothing below 2**-39 of the largest
counts) and multiplied by w and x.
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
    yield
    assert sg.linear_timeouts() == 0


def reference(x, w, targets):
    """(loss, lse, bound of both, z, zb)"""
    M, N, K = x.shape[0], w.shape[1], x.shape[1]
    z = x.double() @ w.double()
    zb = L.product_bound(K, x.double().abs() @ w.double().abs(), x.dtype)
    lse = torch.logsumexp(z, 1)
    adds = 2 * (16 + 8 + N / 512)
    high = z.amax(1) if N else z.new_zeros(M)
    bound = (zb.amax(1) if N else z.new_zeros(M)) + 2.0 ** -21 + adds * U + 4 * U * (high.abs() + lse.abs() + 1)
    some = (targets >= 0) & (targets < N)
    hit = z.gather(1, targets.clamp(0, max(N - 1, 0)).long()[:, None])[:, 0] if N else z.new_zeros(M)
    loss = torch.where(some, lse - hit, torch.zeros_like(lse))
    return loss, lse, torch.where(some, 2 * bound + 2 * U * hit.abs(), torch.zeros_like(bound)), bound, z, zb


def check_forward(x, w, targets):
    loss, lse = sg.linear_cross_entropy(x, w, targets)
    want, want_lse, lb, eb, z, zb = reference(x, w, targets)
    assert loss.dtype == lse.dtype == torch.float32
    L.assert_within(lse, want_lse, eb, "lse")
    L.assert_within(loss, want, lb, "loss")
    return loss, lse, z, zb


def check_backward(x, w, targets, lse, z, zb, dloss, dlse=None):
    dx, dw = sg.linear_cross_entropy_backward(dloss, x, w, targets, lse, dlse=dlse)
    assert dw.shape == w.shape and dw.stride() == w.stride() or not w.is_contiguous()
    M, N, dtype = x.shape[0], w.shape[1], x.dtype
    some = (targets >= 0) & (targets < N)
    g = torch.where(some, dloss.double(), torch.zeros_like(dloss.double())) if dloss is not None else z.new_zeros(M)
    a = g + dlse.double() if dlse is not None else g
    p = torch.exp(z - lse.double()[:, None])
    dz = p * a[:, None]
    dz[some, targets[some].long()] -= g[some]
    # of p: the logit, the exponent, the exponential; of dz: its rounding
    e = p * a.abs()[:, None] * (zb + 4 * U * (z.abs() + lse.double().abs()[:, None]) + 2.0 ** -21)
    e = e + 4 * U * (dz.abs() + g.abs()[:, None] * (dz - p * a[:, None] != 0))
    if dtype != torch.float32:
        most = torch.maximum(a.abs().max(), g.abs().max()) if M else 0.0
        e = e + L.UNIT[dtype] * (dz.abs() + e) + (most * 2.0 ** -39 if dtype == torch.float16 else 0)
    xd, wd = x.double(), w.double()
    ref = dz @ wd.t()
    # float32: the pieces of the vocabulary are added up in float32
    L.assert_within(dx, ref, e @ wd.abs().t() + L.product_bound(N, (dz.abs() + e) @ wd.abs().t(), dtype) + L.rounding(ref, dtype), "dx")
    ref = xd.t() @ dz
    L.assert_within(dw, ref, xd.abs().t() @ e + L.product_bound(M, xd.abs().t() @ (dz.abs() + e), dtype) + L.rounding(ref, dtype), "dw")
    return dx, dw


def inputs(g, M, N, K, dt, order, pad=0, drop=0.2, wide=torch.int64):
    x = L.strided(g, M, K, dt, pad)
    w = L.weight(g, K, N, dt, order, scale=2 / max(K, 1) ** 0.5)
    targets = torch.randint(0, max(N, 1), (M,), generator=g, device="cuda")
    away = torch.tensor([-100, -1, N, N + 5, 2 ** 31 - 1, -2 ** 31], device="cuda")[torch.randint(0, 6, (M,), generator=g, device="cuda")]
    targets = torch.where(torch.rand((M,), generator=g, device="cuda") < drop, away, targets).to(wide)
    return x, w, targets


SIZES = [(1, 1, 1), (1, 700, 64), (2, 17, 5), (7, 64, 64), (33, 300, 40), (64, 1000, 512), (128, 256, 128), (129, 257, 65),
         (200, 5003, 100), (256, 31, 777), (300, 2048, 264), (1000, 1030, 777)]


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("order", [0, 1])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_loss_and_gradient(dtype, order, M, N, K):
    dt = L.TYPES[dtype]
    g = L.rng(M + N + K + order)
    for pad, wide in ((0, torch.int64), (8, torch.int32), (3, torch.int64)):
        x, w, targets = inputs(g, M, N, K, dt, order, pad, wide=wide)
        loss, lse, z, zb = check_forward(x, w, targets)
        even = torch.full((M,), 1.0 / M, device="cuda")
        check_backward(x, w, targets, lse, z, zb, even)
        check_backward(x, w, targets, lse, z, zb, torch.randn((M,), generator=g, device="cuda") * 1e-3, torch.randn((M,), generator=g, device="cuda") * 1e-4)


@pytest.mark.parametrize("dtype", L.TYPES)
def test_some_gradients(dtype):
    dt = L.TYPES[dtype]
    g = L.rng(1)
    x, w, targets = inputs(g, 100, 600, 96, dt, 1)
    loss, lse, z, zb = check_forward(x, w, targets)
    dloss, dlse = torch.randn((100,), generator=g, device="cuda"), torch.randn((100,), generator=g, device="cuda")
    dx, dw = check_backward(x, w, targets, lse, z, zb, dloss)
    only, none = sg.linear_cross_entropy_backward(dloss, x, w, targets, lse, need_dw=False)
    assert none is None and torch.equal(only, dx)
    none, only = sg.linear_cross_entropy_backward(dloss, x, w, targets, lse, need_dx=False)
    assert none is None and torch.equal(only, dw)
    check_backward(x, w, targets, lse, z, zb, None, dlse)
    dx, dw = check_backward(x, w, targets, lse, z, zb, torch.zeros_like(dloss))
    assert (dx == 0).all() and (dw == 0).all()
    dx, dw = sg.linear_cross_entropy_backward(None, x, w, targets, lse)
    assert (dx == 0).all() and (dw == 0).all()


@pytest.mark.parametrize("dtype", L.TYPES)
def test_large_and_small_logits(dtype):
    # one logit far above the rest, all far below zero, and rows of weights that rule a column out
    dt = L.TYPES[dtype]
    g = L.rng(2)
    x, w, targets = inputs(g, 60, 500, 64, dt, 1, drop=0)
    w = (w.float() * 4).to(dt)
    loss, lse, z, zb = check_forward(x, w, targets)
    check_backward(x, w, targets, lse, z, zb, torch.full((60,), 1 / 60, device="cuda"))
    x[:, 0], w[0] = 100, -3  # every logit 300 lower
    loss, lse, z, zb = check_forward(x, w, targets)
    check_backward(x, w, targets, lse, z, zb, torch.full((60,), 1 / 60, device="cuda"))


def test_small_losses_keep_their_gradients_in_float16():
    # 1e-6 a token: dz itself would vanish in float16
    g = L.rng(3)
    x, w, targets = inputs(g, 64, 3000, 64, torch.float16, 1, drop=0)
    loss, lse, z, zb = check_forward(x, w, targets)
    dx, dw = check_backward(x, w, targets, lse, z, zb, torch.full((64,), 1e-3, device="cuda"))
    small = sg.linear_cross_entropy_backward(torch.full((64,), 1e-6, device="cuda"), x, w, targets, lse)
    check_backward(x, w, targets, lse, z, zb, torch.full((64,), 1e-6, device="cuda"))
    # a thousandth of the larger gradient, up to the two results' roundings: 2**-25 below float16's
    # normal range (at values of 2.7e-7 that is 6 % of them: half a step of 6e-8), 2**-11 of dx
    goal = dx.double() * 1e-3
    assert ((small[0].double() - goal).abs() <= 2.0 ** -25 * 1.01 + 2.0 ** -11 * 1.01 * goal.abs()).all()


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("order", [0, 1])
def test_gradient_in_pieces(dtype, order):
    # more of dz than is made at a time: 2**28 values are 256 columns of 2**20 tokens
    dt = L.TYPES[dtype]
    g = L.rng(4)
    M, N, K = 2 ** 19 + 3, 1300, 16
    x, w, targets = inputs(g, M, N, K, dt, order, drop=0.05)
    loss, lse = sg.linear_cross_entropy(x, w, targets)
    dloss = torch.full((M,), 1.0 / M, device="cuda")
    dx, dw = sg.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    # some tokens' dx by the formula, dw as a sum of parts that take one piece each
    pick = torch.randint(0, M, (500,), generator=g, device="cuda")
    _, want_lse, _, eb, z, zb = reference(x[pick], w, targets[pick])
    L.assert_within(lse[pick], want_lse, eb, "lse")
    want = torch.zeros((K, N), dtype=torch.float64, device="cuda")
    size, rounded = torch.zeros_like(want), torch.zeros_like(want)
    for a in range(0, M, 2 ** 16):
        r = slice(a, a + 2 ** 16)
        zr = x[r].double() @ w.double()
        dz = torch.exp(zr - lse[r].double()[:, None])
        some = (targets[r] >= 0) & (targets[r] < N)
        dz = dz * some[:, None]
        dz[some, targets[r][some]] -= 1
        dz = dz / M
        want += x[r].double().t() @ dz
        size += x[r].double().abs().t() @ dz.abs()
        if a == 0:
            ref = dz @ w.double().t()
            wide = dz.abs() @ w.double().abs().t()
            e = 2e-5 * wide + (L.UNIT[dt] * wide if dt != torch.float32 else 0) + (2.0 ** -39 / M * w.double().abs().sum(1) if dt == torch.float16 else 0)
            L.assert_within(dx[r], ref, e + L.product_bound(N, wide, dt) + L.rounding(ref, dt), "dx")
    # float16: of 524291 / 2**39 nothing is left
    e = 2e-5 * size + (L.UNIT[dt] * size if dt != torch.float32 else 0) + (2.0 ** -39 * 8 if dt == torch.float16 else 0)
    # the tensor cores' additions that cut: half a million of them, each of a block's sum
    L.assert_within(dw, want, e + L.product_bound(M, size, dt) + L.rounding(want, dt), "dw")


def test_nothing_to_sum():
    for dt in L.TYPES.values():
        x, w = torch.ones((4, 8), dtype=dt, device="cuda"), torch.ones((8, 16), dtype=dt, device="cuda")
        t = torch.tensor([1, -1, 5, 16], device="cuda")
        loss, lse = sg.linear_cross_entropy(x[:0], w, t[:0])
        assert loss.shape == (0,) and lse.shape == (0,)
        loss, lse = sg.linear_cross_entropy(x[:, :0], w[:0], t)
        want = torch.log(torch.tensor(16.0))
        assert (lse.cpu() - want).abs().max() < 1e-6 and (loss.cpu() - torch.tensor([want, 0, want, 0])).abs().max() < 1e-6
        loss, lse = sg.linear_cross_entropy(x, w[:, :0], t)
        assert (loss == 0).all() and (lse == -float("inf")).all()
        ones = torch.ones(4, device="cuda")
        dx, dw = sg.linear_cross_entropy_backward(ones[:0], x[:0], w, t[:0], ones[:0])
        assert dx.shape == (0, 8) and (dw == 0).all()
        dx, dw = sg.linear_cross_entropy_backward(ones, x, w[:, :0], t, ones)
        assert (dx == 0).all() and dw.shape == (8, 0)
        dx, dw = sg.linear_cross_entropy_backward(ones, x[:, :0], w[:0], t, ones)
        assert dx.shape == (4, 0) and dw.shape == (0, 16)


def test_not_a_number_stays_in_its_row():
    g = L.rng(5)
    for dt in L.TYPES.values():
        x, w, targets = inputs(g, 40, 200, 32, dt, 1, drop=0)
        x[7, 3] = float("nan")
        loss, lse = sg.linear_cross_entropy(x, w, targets)
        bad = torch.isnan(loss).nonzero().flatten().tolist()
        assert bad == [7] and torch.isnan(lse).nonzero().flatten().tolist() == [7]
        dx, dw = sg.linear_cross_entropy_backward(torch.ones(40, device="cuda"), x, w, targets, lse)
        assert torch.isnan(dx).any(1).nonzero().flatten().tolist() == [7] and torch.isnan(dw).all()


def test_gradient_against_differences():
    g = L.rng(6)
    x, w, targets = inputs(g, 5, 23, 9, torch.float32, 0, drop=0)
    dloss, dlse = torch.randn(5, generator=g, device="cuda"), torch.randn(5, generator=g, device="cuda")
    loss, lse = sg.linear_cross_entropy(x, w, targets)
    dx, dw = sg.linear_cross_entropy_backward(dloss, x, w, targets, lse, dlse=dlse)

    def value(x, w):
        z = x @ w
        s = torch.logsumexp(z, 1)
        return ((s - z.gather(1, targets[:, None])[:, 0]) * dloss.double()).sum() + (s * dlse.double()).sum()

    step = 1e-5
    for t, got, other in ((0, dx, None), (1, dw, None)):
        base = [x.double().clone(), w.double().clone()]
        for i in range(base[t].shape[0]):
            for j in range(base[t].shape[1]):
                up, down = [b.clone() for b in base], [b.clone() for b in base]
                up[t][i, j] += step
                down[t][i, j] -= step
                assert abs((value(*up) - value(*down)) / (2 * step) - got[i, j]) < 2e-5


def test_refusals():
    x, w = torch.ones((4, 8), device="cuda"), torch.ones((8, 16), device="cuda")
    t, f = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.ones(4, device="cuda")
    for call, error in [(lambda: sg.linear_cross_entropy(x, w[:7], t), ValueError), (lambda: sg.linear_cross_entropy(x, w.half(), t), TypeError),
                        (lambda: sg.linear_cross_entropy(x, w, t[:3]), ValueError), (lambda: sg.linear_cross_entropy(x, w, f), TypeError),
                        (lambda: sg.linear_cross_entropy(x, w, t.cpu()), TypeError), (lambda: sg.linear_cross_entropy(x[0], w, t), ValueError),
                        (lambda: sg.linear_cross_entropy(x.double(), w.double(), t), TypeError),
                        (lambda: sg.linear_cross_entropy(x.t(), w, t), ValueError),
                        (lambda: sg.linear_cross_entropy(x, w, torch.zeros(8, dtype=torch.int64, device="cuda")[::2]), ValueError),
                        (lambda: sg.linear_cross_entropy_backward(f[:3], x, w, t, f), ValueError),
                        (lambda: sg.linear_cross_entropy_backward(f, x, w, t, f.half()), TypeError),
                        (lambda: sg.linear_cross_entropy_backward(f, x, w, t, None), ValueError),
                        (lambda: sg.linear_cross_entropy_backward(f, x, w, t, f, dlse=f.double()), TypeError)]:
        with pytest.raises(error):
            call()


# Logits known exactly: 1000 of the target and 992 of the 63 others.  The loss is
# log(1 + 63 e**-8) = 0.0209, whose terms are off by 2**-21 of them and whose sum by at
# most 64 + 16 roundings of about 1: 5e-6.  lse is near 1000, a rounding of it 3e-5.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("tokens", [3, 200])
def test_loss_below_the_rounding_of_lse(dtype, tokens):
    w = torch.eye(64, device="cuda", dtype=dtype)
    targets = torch.arange(tokens, device="cuda") % 64
    x = torch.full((tokens, 64), 992.0, device="cuda", dtype=dtype)
    x[torch.arange(tokens, device="cuda"), targets] = 1000.0
    loss, lse = sg.linear_cross_entropy(x, w, targets)
    want = torch.logsumexp(x.double(), 1) - 1000
    assert float((loss.double() - want).abs().max()) <= 80 * U + 0.0212 * 2.0 ** -21
    assert float((lse.double() - want - 1000).abs().max()) <= 2.0 ** -15 + 80 * U


# Half of the tokens' logits are sums of one sign (the target's weight is in x), where
# additions that are cut off instead of rounded tell most.  dx = dz w^T with p = exp(z - lse):
# a relative 2**-24 (|z| + |lse|) of p for the exponent's rounding, and of z itself the
# products' 2**-22 |z| (three pieces of each operand hold 24 bits; 64 K's worth of largest
# products is cut off four times by at most 2**-23 of the sum), |z| and |lse| at most 40.
@pytest.mark.parametrize("M,N,K", [(90, 74, 1088), (533, 2397, 128), (37, 64, 227)])
def test_gradient_of_large_logits(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M)
    w = torch.randn((N, K), generator=g, device="cuda") * (2 / K ** 0.5)
    targets = torch.randint(0, N, (M,), generator=g, device="cuda")
    x = torch.randn((M, K), generator=g, device="cuda")
    x[::2] += 3 * w[targets[::2]]
    dloss = torch.full((M,), 1.0 / M, device="cuda")
    z = x.double() @ w.double().t()
    assert float(z.abs().max()) < 40
    lse = torch.logsumexp(z, 1).float()
    dx, dw = sg.linear_cross_entropy_backward(dloss, x, w.t(), targets, lse)
    p = torch.exp(z - lse.double()[:, None])
    dz = p.clone()
    dz[torch.arange(M), targets] -= 1
    dz /= M
    pb = p / M * (2.0 ** -24 * (2 * 40 + 8) + 2.0 ** -22 * z.abs() + 2.0 ** -22)
    pb[torch.arange(M), targets] += 2.0 ** -23 / M
    S = pb @ w.double().abs()
    A = dz.abs() @ w.double().abs()
    err = (dx.double() - dz @ w.double()).norm()
    assert float(err) <= float((S + L.product_bound(N, A, torch.float32)).norm())
