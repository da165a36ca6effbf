"""How exact the logits under linear_cross_entropy are (needs a GB300).

The tensor core cuts its sums off: an instruction (K of 16) leaves them by up to one
unit in the last place, 2**-23 of them, too small.  With factors of one sign that adds up,
n instructions to (n + 1) / 2 of such units of the whole sum at most, and to about
0.18 n on the average (a cut is half a unit, a unit 0.72 x 2**-23 of its value, the running
sum half of the whole).  So sums are added in FP32 registers, rounded to nearest,
after each block of K: of 512 in 16 bits (128 for up to 128 tokens' losses), with n = 32, and
in FP32, whose small products come first in a block, of 64, with n = 4 that count.

All factors here are between 0.5 and 1.5 and the logits near 30: then all of a token's
logits are too small by nearly the same fraction, which shows in its log sum, and in
the gradient of that as a scale of p = exp(z - lse).
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


def inputs(M, N, K, dtype, order):
    g = L.rng(M + N + K + order)
    x = (0.5 + torch.rand((M, K), generator=g, device="cuda")).to(dtype)
    w = ((0.5 + torch.rand((N, K) if order else (K, N), generator=g, device="cuda")) * (30 / K)).to(dtype)
    w = w.t() if order else w
    z = x.double() @ w.double()
    assert float(z.min()) > 15 and float(z.max()) < 45
    return x, w, torch.randint(0, N, (M,), generator=g, device="cuda"), z


def cut(K, dtype, few=False):
    """The largest error of a logit's sum as a fraction of it: its blocks', and half a unit for each of their additions to half of it."""
    block, n = (64, 4) if dtype == torch.float32 else (128, 8) if few else (512, 32)
    return ((n + 1) / 2 + -(-K // block) / 4) * 2.0 ** -23


# At K = 16384 in one block the average would be 0.18 * 1024 units, 6.6e-4 of a logit of 30;
# allowed are 24.5, 9e-5 (few tokens: 36.5, 1.3e-4), and some 4e-6 for the log sum of 64 exponentials.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("order", [0, 1])
@pytest.mark.parametrize("M", [1, 64, 128, 300, 1000])
def test_log_sums_of_a_long_k(dtype, order, M):
    N, K = 64, 16384
    x, w, targets, z = inputs(M, N, K, dtype, order)
    loss, lse = sg.linear_cross_entropy(x, w, targets)
    want = torch.logsumexp(z, 1)
    most = cut(K, dtype, M <= 128)
    bound = most * z.amax(1) + 2.0 ** -21 + 40 * U + 4 * U * want
    assert ((lse.double() - want).abs() <= bound).all()
    # the loss is a difference of two logits' sums, each cut alike
    hit = z.gather(1, targets[:, None])[:, 0]
    assert ((loss.double() - (want - hit)).abs() <= bound + most * hit + 2 * U * hit).all()


def scale_of(got, want):
    return float((got.double() * want).sum() / want.square().sum())


# dz = p rounded to the type: by at most one step / sqrt(12) in the root mean square, a step at most
# 2 UNIT of p.  A token's 64 p and the tokens are rounded apart from one another, so their mean by that over
# sqrt(64 M) times at most 2 for what p differ by; five of it are allowed.  dx and dw are rounded once
# more, each value by itself: nothing in the mean of 16384 x 64.  In one block of K the scale would
# be off by 6.6e-4 in the 16-bit types.  In FP32 the mean over all logits of what is cut counts, 0.36 units
# for each of 2.5 that are cut from the whole sum, 3.2e-6 of p at logits of 30 (the rounding of the blocks' additions is as
# often up as down).  With 128 K a block the second 64's twenty small products would be cut on top
# of the first 64's sum, ten units of the whole more: measured 9e-6 to 1.1e-5, and 1.1e-6 to 1.9e-6 as it is.
@pytest.mark.parametrize("dtype,K", [(torch.bfloat16, 16384), (torch.float16, 16384), (torch.float32, 128), (torch.float32, 1024)])
@pytest.mark.parametrize("order", [0, 1])
@pytest.mark.parametrize("M", [100, 300, 1000])
def test_scale_of_the_gradient(dtype, K, order, M):
    N = 64
    x, w, targets, z = inputs(M, N, K, dtype, order)
    lse = torch.logsumexp(z, 1).float()
    dx, dw = sg.linear_cross_entropy_backward(None, x, w, targets, lse, dlse=torch.ones(M, device="cuda"))
    p = torch.exp(z - lse.double()[:, None])
    # of p: the logit, the exponential, in 16 bits the exponent's rounding; then dz's rounding
    bound = 2.0 ** -21
    if dtype == torch.float32:
        bound += 0.36 * 2.5 * 2.0 ** -23 * float(z.max())
    else:
        bound += cut(K, dtype) * float(z.max()) + 4 * U * 45 + 5 * 2 * (2 * L.UNIT[dtype] / 12 ** 0.5) / (N * M) ** 0.5
    assert abs(scale_of(dx, p @ w.double().t()) - 1) <= bound
    assert abs(scale_of(dw, x.double().t() @ p) - 1) <= bound


# Tokens that the model is sure of: what is left of 1 - p is a hundredth of p, so an error of
# a logit counts a hundred times.  In the 16-bit types all of dz but the target's is rounded once, by
# UNIT at most, and so is dx; the target's is p - 1 with p off by its logit.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,K", [(64, 4096), (200, 8192), (300, 1000)])
def test_gradient_of_sure_tokens(dtype, M, K):
    N = 64
    x, w, targets, z = inputs(M, N, K, dtype, 1)
    x = x.clone()
    # the target's logit some 8 above the others: along what its weight has more than they
    w = w.clone()
    targets = torch.arange(M, device="cuda") % N
    extra = torch.arange(K, device="cuda") % N
    w = w.t().contiguous()
    w[extra, torch.arange(K, device="cuda")] += 16 / K * N / 8
    w = w.t()
    mine = extra[None, :] == targets[:, None]
    x[mine] += 4
    z = x.double() @ w.double()
    lse = torch.logsumexp(z, 1).float()
    p = torch.exp(z - lse.double()[:, None])
    left = 1 - p.gather(1, targets[:, None])[:, 0]
    assert float(left.median()) < 0.05 and float(left.min()) > 1e-5
    dx, _ = sg.linear_cross_entropy_backward(torch.ones(M, device="cuda"), x, w, targets, lse, need_dw=False)
    dz = p.clone()
    dz[torch.arange(M), targets] -= 1
    ref = dz @ w.double().t()
    e = p * (cut(K, dtype) * z + 8 * U * (z.abs() + lse.double().abs()[:, None]) + 2.0 ** -21)
    e[torch.arange(M), targets] += 2 * U
    if dtype != torch.float32:
        e = e + L.UNIT[dtype] * dz.abs() + (2.0 ** -39 if dtype == torch.float16 else 0)
    bound = e @ w.double().abs().t() + L.product_bound(N, dz.abs() @ w.double().abs().t(), dtype) + L.rounding(ref, dtype)
    L.assert_within(dx, ref, bound, "dx")
