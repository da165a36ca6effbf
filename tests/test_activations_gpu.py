"""Activations and their slopes by themselves: the product is zero, so the bias,
or the saved argument, is z.  Through every epilogue (needs a GB300)."""
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


def _arguments(dtype):
    """-12 .. 12, and the ends of the type's range, infinities and a NaN."""
    top = torch.finfo(dtype).max
    ends = [0.0, -0.0, top, -top, top / 2, -top / 2, float("inf"), -float("inf"), float("nan")]
    return torch.cat([torch.linspace(-12, 12, 1200, dtype=torch.float64), torch.tensor(ends, dtype=torch.float64)]).to(dtype).cuda()


# Logistics below the smallest normal number may be 0; times an argument of -12 that is 12 * 2**-126.
FLOOR = 2.0 ** -122

# few tokens, the product kernel with K in one piece and shared out, and without any K
ROUTES = [(2, 40), (40, 40), (150, 40), (80, 4096), (70, 0)]


def _through(z, act, M, K):
    return sg.linear(torch.zeros(M, K, dtype=z.dtype, device="cuda"), torch.zeros(K, z.numel(), dtype=z.dtype, device="cuda"),
                     z, activation=act)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", L.ACTS)
@pytest.mark.parametrize("M,K", ROUTES)
def test_values_16_bit(dtype, act, M, K):
    z = _arguments(L.TYPES[dtype])
    want = L.value(z.double(), act).expand(M, -1)
    L.assert_within(_through(z, act, M, K), want, L.act_bound(want, z.dtype) + L.rounding(want, z.dtype) + FLOOR, f"{act} {dtype} {M} {K}")
