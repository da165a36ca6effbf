"""The statistics that layer_norm saves of rows with a NaN or an infinity, in each of
its forms (needs a GB300): the deviation of such a row is no number, so neither is
what is saved of it, and its mean is not finite."""
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


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("N", [1, 2, 31, 300, 1001, 4096, 4098, 8193, 12289, 16384, 40000])
def test_rows_out_of_range(dtype, N):
    g = L.rng(N)
    x = L.randn(g, (160, N), L.TYPES[dtype])
    bad = {3: float("nan"), 50: float("inf"), 51: -float("inf"), 159: float("nan")}
    for row, value in bad.items():
        x[row, row % N] = value
    if N > 1:
        x[100, 0], x[100, 1] = float("inf"), -float("inf")
        bad[100] = None
    stats = torch.empty((160, 2), device="cuda")
    y = sg.layer_norm(x, stats=stats)
    good = torch.ones(160, dtype=torch.bool, device="cuda")
    good[list(bad)] = False
    assert torch.isfinite(stats[good]).all() and torch.isfinite(y[good]).all()
    assert torch.isnan(stats[~good, 1]).all() and not torch.isfinite(stats[~good, 0]).any()
    assert torch.isnan(y[~good]).any(1).all()
