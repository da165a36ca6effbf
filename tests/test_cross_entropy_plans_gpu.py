"""Every plan of the product kernel under linear_cross_entropy and its gradient
(needs a GB300): LINEAR_TUNE limits the tiles, read once a process."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import torch
import dense_fp32_tiled_gb300 as sg
from tests import _layers as L
from tests.test_cross_entropy_gpu import check_backward, check_forward, inputs
g = L.rng(1)
for dt in L.TYPES.values():
    for order in (0, 1):
        for M, N, K in ((300, 1500, 200), (70, 5000, 96), (520, 700, 1100)):
            x, w, t = inputs(g, M, N, K, dt, order)
            loss, lse, z, zb = check_forward(x, w, t)
            check_backward(x, w, t, lse, z, zb, torch.full((M,), 1.0 / M, device="cuda"))
assert sg.linear_timeouts() == 0
print("all within their bounds")
"""


@pytest.mark.parametrize("tune", [f"cg=1,bt={b}" for b in (16, 32, 64, 96, 128, 160, 192, 224, 256)] +
                         [f"cg=2,bt={b}" for b in (64, 96, 128, 160, 192, 224, 256)])
def test_plan(tune):
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, env=dict(os.environ, LINEAR_TUNE=tune), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all within" in r.stdout, r.stdout[-1000:] + r.stderr[-3000:]
