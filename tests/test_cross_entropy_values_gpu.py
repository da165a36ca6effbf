"""linear_cross_entropy_backward of gradients that are no numbers or infinite, which stay
in their tokens' rows (needs a GB300)."""
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_tiled_gb300 as sg
from tests import _layers as L
from tests.test_cross_entropy_gpu import inputs

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


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("M,N,K", [(40, 300, 64), (1500, 700, 100)])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("where", ["dloss", "dlse"])
def test_one_gradient_out_of_range(dtype, M, N, K, value, where):
    # times 2**14 a float16 of 4 is out of range: of the other tokens' gradients the largest counts
    g = L.rng(M + N)
    x, w, targets = inputs(g, M, N, K, L.TYPES[dtype], 1, drop=0)
    loss, lse = sg.linear_cross_entropy(x, w, targets)
    dloss = torch.randn((M,), generator=g, device="cuda") * 3 + 8
    dlse = torch.randn((M,), generator=g, device="cuda")
    # the bad token's own other gradient is not what the others are measured by
    dloss[7] = dlse[7] = 0
    want, _ = sg.linear_cross_entropy_backward(dloss, x, w, targets, lse, dlse=dlse)
    assert torch.isfinite(want).all()
    (dloss if where == "dloss" else dlse)[7] = value
    dx, dw = sg.linear_cross_entropy_backward(dloss, x, w, targets, lse, dlse=dlse)
    rest = torch.arange(M, device="cuda") != 7
    assert torch.equal(dx[rest], want[rest])
    assert not torch.isfinite(dx[7]).any() and not torch.isfinite(dw).all()


@pytest.mark.parametrize("dtype", L.TYPES)
def test_all_gradients_out_of_range(dtype):
    g = L.rng(9)
    x, w, targets = inputs(g, 5, 40, 16, L.TYPES[dtype], 0, drop=0)
    loss, lse = sg.linear_cross_entropy(x, w, targets)
    for value in (float("inf"), float("nan")):
        dx, dw = sg.linear_cross_entropy_backward(torch.full((5,), value, device="cuda"), x, w, targets, lse)
        assert not torch.isfinite(dx).any() and not torch.isfinite(dw).any()
