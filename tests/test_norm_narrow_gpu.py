"""The gradient of layer norm at rows of at most a pack a lane, whose weights come another
way than those of wider ones (needs a GB300).  Bounds as in test_norm_gpu, but for the columns'
sums: at most 152 blocks of up to 24 rows add a column up, so a thread has M / 152 rows at most,
24 sums are joined in a block and the blocks' by 5 additions and 5 exchanges."""
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_tiled_gb300 as sg
from tests import _layers as L
from tests.test_norm_gpu import U, adds, h_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_fp32_tiled_gb300 import build
    build.build()
    sg.load_library()


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("M,N", [(1, 8), (23, 64), (24, 128), (3649, 128), (9001, 256), (20000, 248), (5000, 264), (700, 512), (300, 30)])
@pytest.mark.parametrize("weight,pad", [(True, 0), (False, 0), (True, 8), (True, 3)])
def test_backward(dtype, M, N, weight, pad):
    dt = L.TYPES[dtype]
    g = L.rng(M + N + pad)
    x, dy = L.strided(g, M, N, dt, pad, 0, scale=2.0), L.strided(g, M, N, dt, pad)
    w = L.randn(g, (N,), dt) if weight else None
    stats = torch.empty((M, 2), device="cuda")
    sg.layer_norm(x, w, None, eps=1e-5, stats=stats)
    dx, dw, db = sg.layer_norm_backward(dy, x, w, stats)
    h, mean, rstd = h_of(x, 1e-5)
    gy = dy.double() * (w.double() if weight else 1.0)
    K = adds(N)
    G, GH = gy.abs().mean(1, keepdim=True), (gy * h).abs().mean(1, keepdim=True)
    ref = rstd * (gy - gy.mean(1, keepdim=True) - h * (gy * h).mean(1, keepdim=True))
    bound = rstd * U * (K + 16) * (gy.abs() + 2 * G + 3 * (h.abs() + 2) * (GH + G)) + L.rounding(ref, dt)
    L.assert_within(dx, ref, bound, "dx")
    chain = M / 152 + 24 + 10
    hb = (K + 8) * U * (h.abs() + 2)
    ref = (dy.double() * h).sum(0)
    L.assert_within(dw, ref, chain * U * (dy.double() * h).abs().sum(0) + (dy.double().abs() * hb).sum(0) + L.rounding(ref, dt), "dweight")
    ref = dy.double().sum(0)
    L.assert_within(db, ref, chain * U * dy.double().abs().sum(0) + L.rounding(ref, dt), "dbias")
    none, dw2, db2 = sg.layer_norm_backward(dy, x, w, stats, need_dx=False)
    assert none is None and torch.equal(dw2, dw) and torch.equal(db2, db)
