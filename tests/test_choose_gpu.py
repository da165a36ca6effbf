"""expert_choose and its gradient against the definition in 64 bits (needs a GB300).

Bounds, in units u = 2**-24 of FP32.  A weight is an exponential (4 u, and the
rounding of its argument, |l - max| u), a quotient (1) by a sum of exponentials
(the same again, and 36 additions at most) and a scale (1): (64 + 2 R) u of it,
R the largest |l - max|.  A gradient p (g - mean) has that error twice, on
|g| + mean |g|, and is rounded to the logits' type.
"""
import math

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


def scores(l, scoring):
    if scoring == "sigmoid":
        e = torch.exp(-l.abs())
        return torch.where(l < 0, e / (1 + e), 1 / (1 + e))
    return torch.softmax(l, 1)


def choice(l, bias, J, scoring, groups, kept, top):
    """chosen by the definition, a stable sort for each step; l in 64 bits."""
    T, E = l.shape
    never = torch.full_like(l, -math.inf)
    v = scores(l, scoring)
    if bias is not None:
        v = v + bias
    allowed = (l > -math.inf) & (v > -math.inf)
    order = torch.where(allowed, l if bias is None else v, never)
    if groups > 1:
        by = order if bias is None and top == 1 else torch.where(allowed, v, never)
        best = by.view(T, groups, -1).sort(dim=2, descending=True).values[:, :, :top]
        total = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2)
        total = torch.where(best[:, :, 0] > -math.inf, total, torch.full_like(total, -math.inf))
        at = total.sort(dim=1, descending=True, stable=True).indices[:, :kept]
        stay = torch.zeros_like(total, dtype=torch.bool).scatter(1, at, True)
        order = torch.where(stay.repeat_interleave(E // groups, 1), order, never)
    value, at = order.sort(dim=1, descending=True, stable=True)
    chosen = torch.where(value > -math.inf, at, torch.full_like(at, -1))[:, :J]
    bad = torch.isnan(l).any(1) | ((scoring == "softmax") & (l == math.inf).any(1))
    chosen[bad] = -1
    return chosen.to(torch.int32)


def weight(l, chosen, scoring, renormalize, scale):
    """(weights, the range of the logits that enter) in 64 bits."""
    some = chosen >= 0
    mine = torch.gather(l, 1, chosen.clamp(min=0).long())
    if scoring == "softmax":
        full = torch.softmax(torch.where(some, mine, torch.full_like(mine, -math.inf)), 1) if renormalize else torch.gather(torch.softmax(l, 1), 1, chosen.clamp(min=0).long())
    else:
        full = torch.where(some, scores(mine, scoring), torch.zeros_like(mine))
        if renormalize:  # by the scores' logarithms: scores of logits below -745 are 0 in 64 bits too, their shares are not
            log = torch.minimum(mine, torch.zeros_like(mine)) - torch.log1p(torch.exp(-mine.abs()))
            full = torch.softmax(torch.where(some, log, torch.full_like(log, -math.inf)), 1)
    return torch.where(some, full, torch.zeros_like(full)) * scale


def reach(l):
    finite = torch.where(torch.isfinite(l), l, torch.zeros_like(l))
    return finite.amax(1, keepdim=True) - finite.amin(1, keepdim=True) + finite.abs().amax(1, keepdim=True)


def check(logits, J, bias=None, scoring="softmax", groups=1, kept=1, top=1, renormalize=True, scale=1.0):
    chosen, w = sg.expert_choose(logits, J, bias=bias, scoring=scoring, groups=groups, kept_groups=kept, group_top=top,
                                 renormalize=renormalize, scale=scale)
    l = logits.double()
    want = choice(l, None if bias is None else bias.double(), J, scoring, groups, kept, top)
    assert chosen.dtype == torch.int32 and w.dtype == torch.float32
    assert torch.equal(chosen, want), f"{int((chosen != want).any(1).sum())} of {len(want)} tokens differ"
    ref = weight(l, want, scoring, renormalize, scale)
    ref[torch.isnan(l).any(1)] = math.nan
    if scoring == "softmax":
        ref[(l == math.inf).any(1)] = math.nan
    L.assert_within(w, ref, (64 + 2 * reach(l)) * U * ref.abs() + 2.0 ** -126, "weights")
    return chosen, w


def some_logits(g, T, E, dtype, pad=0, scale=1.5):
    return L.strided(g, T, E, torch.float32, pad, scale=scale).to(dtype) if not pad else L.strided(g, T, E, dtype, pad, scale=scale)


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("T,E,J", [(1, 1, 1), (1, 16, 2), (3, 7, 7), (5, 33, 5), (129, 64, 8), (1000, 100, 6), (257, 256, 8),
                                   (40, 511, 40), (33, 1000, 64), (20, 1024, 64)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_choice(dtype, T, E, J, scoring):
    g = L.rng(T * 1000 + E)
    logits = some_logits(g, T, E, L.TYPES[dtype], pad=(0, 3)[E % 2])
    for renormalize, scale in ((True, 1.0), (False, 2.5)):
        check(logits, J, scoring=scoring, renormalize=renormalize, scale=scale)
        bias = torch.randn((E,), generator=g, device="cuda") * 0.05
        check(logits, J, bias=bias, scoring=scoring, renormalize=renormalize, scale=scale)


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("E,groups,kept,J", [(256, 8, 4, 8), (60, 3, 1, 6), (64, 32, 5, 4), (1024, 2, 1, 12), (9, 9, 4, 3), (12, 3, 2, 8)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_groups(dtype, E, groups, kept, J, scoring):
    g = L.rng(E + groups)
    logits = some_logits(g, 300, E, L.TYPES[dtype])
    for top in (1, 2):
        for bias in (None, torch.randn((E,), generator=g, device="cuda") * 0.05):
            check(logits, J, bias=bias, scoring=scoring, groups=groups, kept=kept, top=top)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_equal_values_come_in_order(scoring):
    g = L.rng(3)
    coarse = (torch.randn((400, 64), generator=g, device="cuda") * 2).round() / 2
    for bias in (None, torch.zeros(64, device="cuda"), torch.tensor([0.0, 0.25] * 32, device="cuda")):
        check(coarse, 8, bias=bias, scoring=scoring)
        for top in (1, 2):
            check(coarse, 8, bias=bias, scoring=scoring, groups=8, kept=3, top=top)
    check(torch.zeros((5, 40), device="cuda"), 6, bias=torch.zeros(40, device="cuda"), scoring=scoring, groups=4, kept=2, top=2)
    signed = torch.zeros((3, 40), device="cuda")
    signed[:, ::2] = -0.0
    check(signed, 6, scoring=scoring)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [24, 256, 1000])
def test_values_that_32_bits_cannot_tell_apart(scoring, E):
    # biases that undo the scores to the last bit of FP32: what is left decides, in 64 bits
    g = L.rng(E)
    row = torch.randn((1, E), generator=g, device="cuda")
    v = scores(row.double(), scoring)[0]
    logits = row.expand(50, E).contiguous()
    logits[1:] += torch.randn((49, E), generator=g, device="cuda") * 1e-6  # other tokens: close, but not so close
    for level in (1.0, 0.0, 100.0):
        bias = (level - v).float()
        check(logits, 8, bias=bias, scoring=scoring)
        check(logits, 8, bias=bias, scoring=scoring, groups=E // 8 if E == 24 else 4, kept=2, top=2)


def test_groups_whose_best_two_are_equal_sums_in_32_bits():
    g = L.rng(8)
    logits = torch.randn((64, 32), generator=g, device="cuda")
    logits[:, 8:16] = logits[:, 0:8].flip(1) + torch.randn((64, 8), generator=g, device="cuda") * 1e-7
    check(logits, 4, scoring="sigmoid", groups=4, kept=1, top=2)
    check(logits, 4, scoring="softmax", groups=4, kept=2, top=2)


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_masked_experts_and_tokens(dtype, scoring):
    g = L.rng(4)
    dt = L.TYPES[dtype]
    logits = some_logits(g, 64, 40, dt)
    logits[torch.rand((64, 40), generator=g, device="cuda") < 0.9] = -math.inf  # few are left, sometimes none
    logits[7] = -math.inf
    logits[8] = torch.finfo(dt).min                                             # the type's lowest value is a value
    logits[9, 1:] = torch.finfo(dt).min
    bias = torch.randn((40,), generator=g, device="cuda")
    bias[3] = -math.inf
    for b in (None, bias):
        for renormalize in (True, False):
            chosen, w = check(logits, 6, bias=b, scoring=scoring, renormalize=renormalize)
            check(logits, 6, bias=b, scoring=scoring, renormalize=renormalize, groups=5, kept=2, top=2)
            assert (chosen[7] == -1).all() and (w[7] == 0).all()
            assert b is None or not (chosen == 3).any()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_not_a_number_and_infinity(scoring):
    g = L.rng(5)
    logits = torch.randn((6, 40), generator=g, device="cuda")
    logits[1, 7] = math.nan
    logits[3, 9] = math.inf
    logits[4, 2] = math.nan
    logits[4, 3] = math.inf
    bias = torch.randn((40,), generator=g, device="cuda") * 0.1
    for b in (None, bias):
        chosen, w = check(logits, 5, bias=b, scoring=scoring)
        assert (chosen[1] == -1).all() and torch.isnan(w[1]).all()
    bias[4] = math.nan  # an expert with no bias to compare by
    chosen, _ = sg.expert_choose(logits[:1], 40, bias=bias, scoring=scoring)
    assert 4 not in chosen[0, :39].tolist() and chosen[0, 39] == -1


def test_small_scores_keep_their_shares():
    # chosen by the bias, with scores far below the largest: renormalised they are still their shares
    logits = torch.full((2, 10), 0.0, device="cuda")
    logits[:, 5:] = -200.0 + torch.arange(5, device="cuda") * 0.5
    bias = torch.zeros(10, device="cuda")
    bias[5:] = 3.0
    for scoring in ("softmax", "sigmoid"):
        _, w = check(logits, 4, bias=bias, scoring=scoring)
        assert (w.sum(1) - 1).abs().max() < 1e-6


def gradient(l, chosen, dw, scoring, renormalize, scale):
    """(dlogits, the size of what it is a difference of) by the formulas."""
    T, E = l.shape
    some = chosen >= 0
    at = chosen.clamp(min=0).long()
    p = weight(l, chosen, scoring, renormalize, 1.0)
    g = torch.where(some, dw.double() * scale, torch.zeros_like(p))
    mean, mabs = (p * g).sum(1, keepdim=True), (p * g.abs()).sum(1, keepdim=True)
    put = lambda x: torch.zeros((T, E), dtype=torch.float64, device=l.device).scatter_add_(1, at, torch.where(some, x, torch.zeros_like(x)))
    far = 1 - torch.where(some, scores(torch.gather(l, 1, at), "sigmoid"), torch.zeros_like(p)) if scoring == "sigmoid" else None
    if scoring == "softmax" and not renormalize:
        full = torch.where(some.any(1, keepdim=True), torch.softmax(l, 1), torch.zeros_like(l))
        return full * (put(g) - mean), full * (put(g.abs()) + mabs)
    if scoring == "softmax":
        return put(p * (g - mean)), put(p * (g.abs() + mabs))
    if renormalize:
        return put(p * far * (g - mean)), put(p * far * (g.abs() + mabs))
    return put(p * far * g), put(p * far * g.abs())


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,J", [(1, 1, 1), (3, 7, 7), (5, 33, 5), (129, 64, 8), (1000, 100, 6), (40, 511, 40), (33, 1000, 64)])
def test_gradient(dtype, scoring, renormalize, T, E, J):
    g = L.rng(T + E)
    logits = some_logits(g, T, E, L.TYPES[dtype], pad=(0, 3)[E % 2])
    if T > 2:
        logits[1, : E // 2] = -math.inf
        logits[2] = -math.inf
    chosen, _ = sg.expert_choose(logits, J, scoring=scoring)
    dw = torch.randn((T, J), generator=g, device="cuda")
    got = sg.expert_choose_backward(dw, logits, chosen, scoring=scoring, renormalize=renormalize, scale=1.5)
    l = logits.double()
    ref, size = gradient(l, chosen, dw, scoring, renormalize, 1.5)
    assert got.dtype == logits.dtype
    L.assert_within(got, ref, (150 + 4 * reach(l)) * U * size + L.rounding(ref, logits.dtype) + 2.0 ** -126, "dlogits")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_against_differences(scoring, renormalize):
    g = L.rng(11)
    logits = torch.randn((4, 20), generator=g, device="cuda")
    chosen, _ = sg.expert_choose(logits, 5, scoring=scoring)
    dw = torch.randn((4, 5), generator=g, device="cuda")
    got = sg.expert_choose_backward(dw, logits, chosen, scoring=scoring, renormalize=renormalize, scale=2.0).double()
    h = 1e-5  # in 64 bits: differences are within 1e-10 + 1e-16 / h
    for e in range(20):
        step = torch.zeros((1, 20), dtype=torch.float64, device="cuda")
        step[0, e] = h
        up = weight(logits.double() + step, chosen, scoring, renormalize, 2.0)
        down = weight(logits.double() - step, chosen, scoring, renormalize, 2.0)
        slope = ((up - down) * dw.double()).sum(1) / (2 * h)
        assert (got[:, e] - slope).abs().max() < 1e-5


def test_gradient_of_choices_given_twice_and_of_none():
    g = L.rng(12)
    logits = torch.randn((3, 20), generator=g, device="cuda")
    chosen = torch.tensor([[4, 4, 9], [-1, 3, 25], [-1, -1, -1]], dtype=torch.int32, device="cuda")
    dw = torch.randn((3, 3), generator=g, device="cuda")
    got = sg.expert_choose_backward(dw, logits, chosen, scoring="sigmoid", renormalize=False).double()
    s = scores(logits.double(), "sigmoid")
    want = torch.zeros_like(s)
    want[0, 4], want[0, 9], want[1, 3] = dw[0, 0] + dw[0, 1], dw[0, 2], dw[1, 1]
    assert (got - want * s * (1 - s)).abs().max() < 1e-6


def test_empty_and_refused():
    g = L.rng(13)
    logits = torch.randn((4, 8), generator=g, device="cuda")
    chosen, w = sg.expert_choose(logits[:0], 2)
    assert chosen.shape == (0, 2) and w.shape == (0, 2)
    chosen, w = sg.expert_choose(logits, 0)
    assert chosen.shape == (4, 0)
    assert (sg.expert_choose_backward(w, logits, chosen) == 0).all()
    for call, error in [(lambda: sg.expert_choose(logits, 9), sg.SgemmError), (lambda: sg.expert_choose(logits, -1), sg.SgemmError),
                        (lambda: sg.expert_choose(logits, 2, groups=3), sg.SgemmError),
                        (lambda: sg.expert_choose(logits, 2, groups=2, kept_groups=3), sg.SgemmError),
                        (lambda: sg.expert_choose(logits, 2, groups=2, group_top=3), sg.SgemmError),
                        (lambda: sg.expert_choose(logits, 2, scoring="relu"), ValueError),
                        (lambda: sg.expert_choose(logits, 2, bias=logits[0].double()), TypeError),
                        (lambda: sg.expert_choose(logits, 2, bias=logits[0, :7]), ValueError),
                        (lambda: sg.expert_choose(logits.t(), 2), ValueError),
                        (lambda: sg.expert_choose(logits[0], 2), ValueError),
                        (lambda: sg.expert_choose(logits.cpu(), 2), TypeError),
                        (lambda: sg.expert_choose(torch.zeros((2, 1025), device="cuda"), 2), sg.SgemmError),
                        (lambda: sg.expert_choose_backward(w, logits, chosen.long()), TypeError),
                        (lambda: sg.expert_choose_backward(torch.zeros((4, 2), device="cuda"), logits, chosen), ValueError),
                        (lambda: sg.expert_choose_backward(None, logits, chosen), ValueError)]:
        with pytest.raises(error):
            call()


def test_the_choice_goes_to_the_experts():
    # with the sort and the way back: tokens without experts keep their residual
    g = L.rng(14)
    logits = torch.randn((50, 6), generator=g, device="cuda")
    logits[10:20] = -math.inf
    x = torch.randn((50, 32), generator=g, device="cuda")
    chosen, w = sg.expert_choose(logits, 2)
    rows, offsets = sg.expert_sort(chosen, 6)
    y = sg.expert_combine(sg.expert_gather(x, rows, offsets), rows, w, residual=x)
    want = x * 2
    want[10:20] = x[10:20]
    assert int(offsets[-1]) == 80 and (y - want).abs().max() < 1e-5
