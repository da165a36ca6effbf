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

def _value(z, act):
    """L.value, with gelu_tanh as z times a logistic: 1 + tanh is 0 in 64 bits from z = -7.5 on, the product is not."""
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return L.value(z, act)


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
    want = _value(z.double(), act).expand(M, -1)
    L.assert_within(_through(z, act, M, K), want, L.act_bound(want, z.dtype) + L.rounding(want, z.dtype) + FLOOR, f"{act} {dtype} {M} {K}")


def _relative_f32(z, act):
    """Relative error of an FP32 activation evaluated in FP32: the functions' stated errors (erfcf 4 units in
    the last place, expf 2) with four roundings beside them, and for gelu_tanh the six roundings of the
    logistic's argument u, which that multiplies by |u|."""
    base = 2.0 ** -21 + 2.0 ** -22
    if act == "gelu_tanh":
        u = 2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3).abs()
        return base + 6 * 2.0 ** -24 * torch.where(z < 0, u, torch.zeros_like(u)).clamp(max=200)
    return torch.full_like(z, 0.0 if act in ("none", "relu") else base)


@pytest.mark.parametrize("act", L.ACTS)
@pytest.mark.parametrize("M,K", ROUTES)
def test_values_f32(act, M, K):
    z = _arguments(torch.float32)
    want = _value(z.double(), act)
    bound = (_relative_f32(z.double(), act) * want.abs() + FLOOR).expand(M, -1)
    L.assert_within(_through(z, act, M, K), want.expand(M, -1), bound, f"{act} {M} {K}")


def _slopes(z, act):
    """The slope itself: the bias gradient of one row with dy = 1."""
    one = torch.ones(1, z.numel(), dtype=z.dtype, device="cuda")
    x, w = torch.zeros(1, 8, dtype=z.dtype, device="cuda"), torch.zeros(8, z.numel(), dtype=z.dtype, device="cuda")
    return sg.linear_backward(one, x, w, preact=z[None], activation=act, need_dx=False, need_dw=False)[2]


def test_slope_of_gelu_f32():
    """Phi(z) as the value's, z phi(z) with the rounding of z^2 / 2 (times itself) and six more, and their sum."""
    z = _arguments(torch.float32)
    zd = z.double()
    want = L.slope(zd, "gelu")
    cdf, density = 0.5 * torch.erfc(-zd * 0.5 ** 0.5), (zd * torch.exp(-0.5 * zd * zd) * 0.3989422804014327).abs()
    bound = 1.5 * 2.0 ** -21 * cdf + (zd * zd / 2 * 2.0 ** -24 + 2.0 ** -21).clamp(max=1) * density + 2.0 ** -24 * want.abs() + FLOOR
    L.assert_within(_slopes(z, "gelu"), want, bound, "slope of gelu")


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("act", L.ACTS)
def test_slopes(dtype, act):
    """Every activation's, to the ends of the type's range: terms of at most |slope| + 1, each within act_bound."""
    z = _arguments(L.TYPES[dtype])
    want = L.slope(z.double(), act)
    got = _slopes(z, act) if act != "none" else torch.ones_like(z)
    L.assert_within(got, want, L.act_bound(1 + want.abs(), z.dtype) + L.rounding(want, z.dtype) + FLOOR, f"slope of {act} {dtype}")
