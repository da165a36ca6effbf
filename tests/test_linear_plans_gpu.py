"""Every plan of the layer products -- CTA pairs and single CTAs, each tile
width, K split over clusters -- against the formulas in 64 bits, each in a child
process (LINEAR_TUNE is read once), and a few shapes large enough that the
library picks the wide ones itself (needs a GB300)."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import dense_fp32_tiled_gb300 as sg
from tests import _layers as L

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_fp32_tiled_gb300 import build
    build.build()
    sg.load_library()


def check_plan():
    """Dense and by expert, forward and backward, all types, with more tiles than one wave."""
    for dtype in L.TYPES.values():
        g = L.rng(21)
        for M, N, K, order in ((300, 392, 333, 1), (530, 264, 136, 0)):
            x, w, b = L.randn(g, (M, K), dtype), L.weight(g, K, N, dtype, order), L.randn(g, (N,), dtype, 0.5)
            r, z = L.randn(g, (M, N), dtype), torch.empty((M, N), dtype=dtype, device="cuda")
            y, yb, zr, zb = L.forward_ref(x, w, b, r, "silu")
            L.assert_within(sg.linear(x, w, b, r, "silu", preact=z), y, yb, "y")
            L.assert_within(z, zr, zb, "z")
            dy = L.randn(g, (M, N), dtype, 0.5)
            for name, t, (ref, bound) in zip(("dx", "dw", "dbias"), sg.linear_backward(dy, x, w, z, "silu"),
                                             L.backward_ref(dy, x, w, z, "silu")):
                L.assert_within(t, ref, bound, name)
        counts = [5, 0, 200, 64, 33]
        off, at, K, N = L.offsets_of(counts), L.offsets_of(counts).tolist(), 200, 136
        R = sum(counts) + 9
        x, dy, w = L.randn(g, (R, K), dtype), L.randn(g, (R, N), dtype, 0.5), L.weight(g, K, N, dtype, 1, (5,))
        x[at[-1]:] = float("nan")
        dy[at[-1]:] = float("nan")
        got = sg.expert_linear(x, w, off, activation="relu")
        dx, dw, db = sg.expert_linear_backward(dy, x, w, off)
        assert (got[at[-1]:] == 0).all() and (dx[at[-1]:] == 0).all() and (dw[1] == 0).all()
        for e in (0, 2, 3, 4):
            s = slice(at[e], at[e + 1])
            y, yb, _, _ = L.forward_ref(x[s], w[e], None, None, "relu")
            L.assert_within(got[s], y, yb, f"expert {e}")
            for name, t, (ref, bound) in zip(("dx", "dw", "dbias"), (dx[s], dw[e], db[e]), L.backward_ref(dy[s], x[s], w[e], None, "none")):
                L.assert_within(t, ref, bound, f"{name} of expert {e}")
    assert sg.linear_timeouts() == 0


PLANS = [f"cg=2,bt={bt}" for bt in (64, 96, 128, 160, 192, 224, 256)] + \
        [f"cg=1,bt={bt},splits=1" for bt in (16, 32, 64, 96, 128, 160, 192, 224, 256)] + \
        [f"cg=1,bt={bt},splits={s}" for bt, s in ((16, 4), (32, 2), (64, 3), (96, 2), (128, 4))]


@pytest.mark.parametrize("plan", PLANS)
def test_plan(plan):
    code = "import sys; sys.path.insert(0, %r); from tests.test_linear_plans_gpu import check_plan; check_plan()" % ROOT
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=dict(os.environ, LINEAR_TUNE=plan), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-1000:] + r.stderr[-3000:]


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("M,N,K", [(2500, 2100, 333), (4096, 1024, 1024)])
def test_many_waves(dtype, M, N, K):
    dt = L.TYPES[dtype]
    g = L.rng(22)
    x, w, r = L.randn(g, (M, K), dt), L.weight(g, K, N, dt, 1), L.randn(g, (M, N), dt)
    z = torch.empty((M, N), dtype=dt, device="cuda")
    y, yb, zr, zb = L.forward_ref(x, w, None, r, "gelu_tanh")
    L.assert_within(sg.linear(x, w, residual=r, activation="gelu_tanh", preact=z), y, yb, "y")
    L.assert_within(z, zr, zb, "z")
    dy = L.randn(g, (M, N), dt, 0.5)
    for name, t, (ref, bound) in zip(("dx", "dw", "dbias"), sg.linear_backward(dy, x, w, z, "gelu_tanh"),
                                     L.backward_ref(dy, x, w, z, "gelu_tanh")):
        L.assert_within(t, ref, bound, name)


def test_rows_past_32_bits():
    """A result whose elements' offsets pass 2**31, and a row stride that does."""
    g = L.rng(23)
    M, N, K = 70000, 32768, 32
    x, w = L.randn(g, (M, K), torch.bfloat16), L.weight(g, K, N, torch.bfloat16, 1)
    y = sg.linear(x, w)
    ref, bound, _, _ = L.forward_ref(x[-300:], w, None, None, "none")
    L.assert_within(y[-300:], ref, bound, "last rows")
    del y
    out = torch.empty((3, 2 ** 30 + 8), dtype=torch.bfloat16, device="cuda")[:, :N]
    sg.linear(x[:3], w, out=out)
    ref, bound, _, _ = L.forward_ref(x[:3], w, None, None, "none")
    L.assert_within(out, ref, bound, "far rows")
    big = torch.empty((40, 2 ** 27 + 8), dtype=torch.bfloat16, device="cuda")[:, :N]
    sg.linear(x[:40], w, residual=None, out=big)
    ref, bound, _, _ = L.forward_ref(x[:40], w, None, None, "none")
    L.assert_within(big, ref, bound, "far rows of a tile")


def test_far_rows_of_a_route():
    """Rows of the experts' batch whose offsets pass 2**31 elements."""
    g = L.rng(24)
    T, J, H = 70000, 8, 4096
    choices = torch.randint(0, 16, (T, J), generator=g, device="cuda")
    rows, offsets = sg.expert_sort(choices, 16)
    x = L.randn(g, (T, H), torch.bfloat16)
    xs = sg.expert_gather(x, rows, offsets)
    assert xs.numel() > 2 ** 31
    at = torch.tensor([0, 1, T // 2, T - 1], device="cuda")
    for j in (0, J - 1):
        assert torch.equal(xs[rows[at, j].long()], x[at])
    y = sg.expert_gather_backward(xs, rows)
    assert torch.equal(y, (x.float() * J).bfloat16())
