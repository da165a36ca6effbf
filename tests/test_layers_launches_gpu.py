"""How many kernels the layer calls launch, and what another stream may see of
them (needs a GB300)."""
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
    yield
    assert sg.linear_timeouts() == 0


def _products(call):
    """The product kernels that a call launches."""
    for _ in range(2):  # a process's first profile may come out empty
        with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
            call()
            torch.cuda.synchronize()
    return sum(e.count for e in prof.key_averages() if "product_kernel" in e.key)


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("order", [0, 1])
@pytest.mark.parametrize("E", [1, 5, 300])
def test_no_rows_over_many_experts(dtype, order, E):
    """Every expert's gradient is zero, in one launch."""
    dt = L.TYPES[dtype]
    dy, x = torch.empty(0, 72, dtype=dt, device="cuda"), torch.empty(0, 40, dtype=dt, device="cuda")
    w = L.weight(L.rng(E), 40, 72, dt, order, (E,))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    for _ in range(2):
        junk = torch.full((E, 72, 40), 7.0, dtype=dt, device="cuda")  # what dw's memory may hold
        del junk
        dx, dw, db = sg.expert_linear_backward(dy, x, w, offsets)
        assert dx.shape == (0, 40) and dw.shape == (E, 40, 72) and (dw == 0).all() and (db == 0).all()
    assert _products(lambda: sg.expert_linear_backward(dy, x, w, offsets)) == 1


@pytest.mark.parametrize("limit,heard", [("splits=8", True), ("cg=1,bt=20", True), ("cg=1,bt=64,splits=4", False), ("", False)])
def test_limits_that_leave_no_plan_are_reported(limit, heard):
    code = ("import torch, dense_fp32_tiled_gb300 as sg; x, w = torch.ones(100, 4096, device='cuda'), torch.ones(4096, 72, device='cuda');"
            "assert (sg.linear(x, w) == 4096).all() and (sg.linear(x, w) == 4096).all()")
    env = {k: v for k, v in os.environ.items() if k != "LINEAR_TUNE"}
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env={**env, **({"LINEAR_TUNE": limit} if limit else {})},
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stderr.count("LINEAR_TUNE leaves no plan") == int(heard)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_another_stream_behind_an_event_sees_both_products(dtype):
    """An event recorded after a backward pass comes after its second product, which waits for its first."""
    g, dt = L.rng(5), L.TYPES[dtype]
    x, dy = L.randn(g, (4096, 2048), dt), L.randn(g, (4096, 1024), dt)
    w = L.weight(g, 2048, 1024, dt, 1)
    want = [t.clone() for t in sg.linear_backward(dy, x, w)]
    side, event = torch.cuda.Stream(), torch.cuda.Event()
    for _ in range(20):
        got = sg.linear_backward(dy, x, w)
        event.record()
        side.wait_event(event)
        with torch.cuda.stream(side):
            copies = [t.clone() for t in got]
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(copies, want))
