"""expert_choose with a bias where the last pick and the first expert left out are equal,
and others behind both are so near that 32 bits do not tell them apart (needs a GB300).

The choice is exact: that of scores in 64 bits.  Where those are equal too, the definition
itself does not depend on how they are rounded: the sizes below keep scores of different
logits at least some units of 64 bits apart."""
import math

import pytest

torch = pytest.importorskip("torch")

import dense_fp32_tiled_gb300 as sg
from tests import _layers as L
from tests.test_choose_gpu import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_fp32_tiled_gb300 import build
    build.build()
    sg.load_library()


def chosen_of(logits, J, **kw):
    logits = torch.tensor([logits], device="cuda") if isinstance(logits, list) else logits
    return check(logits, J, bias=torch.zeros(logits.shape[1], device="cuda"), **kw)[0][0].tolist()


@pytest.mark.parametrize("dtype", L.TYPES)
def test_a_larger_one_behind_equal_ones(dtype):
    dt = L.TYPES[dtype]
    # sigmoid: 1 in 32 bits for all three
    assert chosen_of(torch.tensor([[17.0, 17.0, 18.0]], device="cuda").to(dt), 1, scoring="sigmoid") == [2]
    # softmax: 0 in 32 bits for all but the first
    assert chosen_of(torch.tensor([[0.0, -200.0, -200.0, -150.0]], device="cuda").to(dt), 2) == [0, 3]


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("E", [40, 100, 256, 1000])
@pytest.mark.parametrize("same", [2, 5, 33])  # 33: more than are brought together
def test_anywhere_in_a_row(dtype, E, same):
    g = L.rng(E + same)
    for scoring, low, high, far in (("sigmoid", 17.0, 18.0, 1.0), ("softmax", -200.0, -150.0, -300.0)):
        logits = torch.full((60, E), far, device="cuda", dtype=L.TYPES[dtype])
        places = torch.rand((60, E), generator=g, device="cuda").argsort(1)
        logits.scatter_(1, places[:, :same], low)
        logits.scatter_(1, places[:, same:same + 1], high)
        logits.scatter_(1, places[:, same + 1:same + 2], 30.0 if scoring == "sigmoid" else 0.0)
        for J in (1, 2, 3):
            chosen, _ = check(logits, J, bias=torch.zeros(E, device="cuda"), scoring=scoring)
            if J >= 2:
                assert torch.equal(chosen[:, 1], places[:, same].int())


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("E,J", [(7, 3), (64, 8), (256, 8), (256, 40), (1000, 64)])
def test_few_different_values(dtype, E, J):
    # logits of ten values whose scores are 1 (or 0) in 32 bits, each of them often
    g = L.rng(E * J)
    steps = torch.randint(0, 10, (300, E), generator=g, device="cuda")
    bias = (torch.randint(0, 2, (E,), generator=g, device="cuda") * 2.0 ** -20).float()
    for logits, scoring in ((17 + steps * 0.5, "sigmoid"), (-100 - 10.0 * steps, "softmax")):
        logits = logits.to(L.TYPES[dtype])
        logits[:, 0] = logits[:, 0] if scoring == "sigmoid" else 0
        check(logits, J, bias=torch.zeros(E, device="cuda"), scoring=scoring)
        check(logits, J, bias=bias, scoring=scoring)
        if E == 256:
            for kept in (1, 4):
                check(logits, J, bias=torch.zeros(E, device="cuda"), scoring=scoring, groups=8, kept=kept, top=2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_equal_ones_with_others_ruled_out(scoring):
    # what is near but masked, or of a group that does not compete, decides nothing
    logits = torch.full((1, 64), 17.0 if scoring == "sigmoid" else -200.0, device="cuda")
    logits[0, 0] = 20.0
    logits[0, 40] = 18.0 if scoring == "sigmoid" else -150.0
    logits[0, 41] = -math.inf
    bias = torch.zeros(64, device="cuda")
    assert check(logits, 2, bias=bias, scoring=scoring)[0][0].tolist() == [0, 40]
    assert check(logits, 2, bias=bias, scoring=scoring, groups=2, kept=1, top=1)[0][0].tolist() == [0, 1]
    bias[40] = -math.inf
    assert check(logits, 2, bias=bias, scoring=scoring)[0][0].tolist() == [0, 1]
