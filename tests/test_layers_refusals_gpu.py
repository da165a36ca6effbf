"""The Python wrappers' refusals on CUDA tensors, through the extension's way
and the interpreter's, and that both ways give the same bits (needs a GB300)."""
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_tiled_gb300 as sg
from dense_fp32_tiled_gb300 import _layers
from tests import _layers as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_fp32_tiled_gb300 import build
    build.build()
    sg.load_library()


@pytest.fixture(params=["extension", "interpreter"])
def way(request, monkeypatch):
    _layers._load()
    if request.param == "extension":
        assert _layers._fast is not None
    else:
        monkeypatch.setattr(_layers, "_fast", None)
    return request.param


def _t(*shape, dtype=torch.bfloat16):
    return torch.ones(shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("call,error", [
    (lambda: sg.linear(_t(4, 8), _t(9, 16)), ValueError),
    (lambda: sg.linear(_t(4, 8), _t(8, 16, dtype=torch.float16)), TypeError),
    (lambda: sg.linear(_t(4, 8, dtype=torch.float64), _t(8, 16, dtype=torch.float64)), TypeError),
    (lambda: sg.linear(_t(4, 8), _t(8, 16).cpu()), TypeError),
    (lambda: sg.linear(_t(2, 4, 8), _t(8, 16)), ValueError),
    (lambda: sg.linear(_t(4, 8), _t(8, 16), activation="swish"), ValueError),
    (lambda: sg.linear(_t(8, 4).t(), _t(8, 16)), ValueError),
    (lambda: sg.linear(_t(4, 8), _t(16, 32)[::2, ::2]), ValueError),
    (lambda: sg.linear(_t(4, 8), _t(8, 1).expand(8, 16)), ValueError),
    (lambda: sg.linear(_t(4, 8), _t(8, 16), bias=_t(15)), ValueError),
    (lambda: sg.linear(_t(4, 8), _t(8, 16), bias=_t(32)[::2]), ValueError),
    (lambda: sg.linear(_t(4, 8), _t(8, 16), bias=_t(16, dtype=torch.float32)), TypeError),
    (lambda: sg.linear(_t(4, 8), _t(8, 16), residual=_t(4, 15)), ValueError),
    (lambda: sg.linear(_t(4, 8), _t(8, 16), preact=_t(5, 16)), ValueError),
    (lambda: sg.linear(_t(4, 8), _t(8, 16), out=_t(4, 17)), ValueError),
    (lambda: (lambda x: sg.linear(x, _t(8, 8), out=x))(_t(4, 8)), sg.SgemmError),
    (lambda: sg.linear_backward(_t(4, 16), _t(4, 8), _t(8, 16), activation="silu"), ValueError),
    (lambda: sg.linear_backward(_t(4, 16), _t(4, 8), _t(8, 16), preact=_t(4, 16)), ValueError),
    (lambda: sg.linear_backward(_t(4, 15), _t(4, 8), _t(8, 16)), ValueError),
    (lambda: sg.expert_linear(_t(4, 8), _t(2, 8, 16), _t(3, dtype=torch.int64)), TypeError),
    (lambda: sg.expert_linear(_t(4, 8), _t(2, 8, 16), _t(2, dtype=torch.int32)), ValueError),
    (lambda: sg.expert_linear(_t(4, 8), _t(8, 16), _t(2, dtype=torch.int32)), ValueError),
    (lambda: sg.expert_linear(_t(4, 8), _t(2, 8, 16), None), ValueError),
    (lambda: sg.expert_linear(_t(4, 8), _t(2, 8, 16), _t(3, dtype=torch.int32), bias=_t(16)), ValueError),
    (lambda: sg.expert_sort(_t(4, 2, dtype=torch.int16), 4), TypeError),
    (lambda: sg.expert_sort(_t(4, dtype=torch.int32), 4), ValueError),
    (lambda: sg.expert_sort(_t(4, 4, dtype=torch.int32).t()[:2], 4), ValueError),
    (lambda: sg.expert_sort(_t(4, 2, dtype=torch.int32), 0), sg.SgemmError),
    (lambda: sg.expert_sort(_t(4, 65, dtype=torch.int32), 4), sg.SgemmError),
    (lambda: sg.expert_gather(_t(4, 8), _t(5, 2, dtype=torch.int32), _t(3, dtype=torch.int32)), ValueError),
    (lambda: sg.expert_combine(_t(8, 8), _t(5, 2, dtype=torch.int32)), ValueError),
    (lambda: sg.expert_combine(_t(10, 8), _t(5, 2, dtype=torch.int32), weights=_t(5, 2)), TypeError),
    (lambda: sg.expert_combine_backward(_t(5, 8), _t(9, 8), _t(5, 2, dtype=torch.int32), None, _t(3, dtype=torch.int32)), ValueError),
])
def test_refusals(way, call, error):
    with pytest.raises(error):
        call()


@pytest.mark.parametrize("dtype", L.TYPES)
def test_both_ways_agree(monkeypatch, dtype):
    _layers._load()
    dt = L.TYPES[dtype]
    g = L.rng(2)
    x, w, b = L.randn(g, (40, 96), dt), L.weight(g, 96, 56, dt, 1), L.randn(g, (56,), dt)
    we, be = L.weight(g, 96, 56, dt, 1, (3,)), L.randn(g, (3, 56), dt)
    dy, z, r = L.randn(g, (40, 56), dt), L.randn(g, (40, 56), dt), L.randn(g, (40, 56), dt)
    off = L.offsets_of([10, 0, 28])
    choices = torch.randint(0, 5, (20, 2), generator=g, device="cuda")
    weights = torch.rand((20, 2), generator=g, device="cuda")

    def run():
        rows, offsets = sg.expert_sort(choices, 5)
        xs = sg.expert_gather(x[:20], rows, offsets)
        return (sg.linear(x, w, b, r, "gelu"), *sg.linear_backward(dy, x, w, preact=z, activation="silu"),
                sg.expert_linear(x, we, off, be, None, "relu"), *sg.expert_linear_backward(dy, x, we, off, need_dbias=True),
                rows, offsets, xs, sg.expert_combine(xs, rows, weights, x[:20]), sg.expert_gather_backward(xs, rows),
                *sg.expert_combine_backward(x[:20], xs, rows, weights, offsets))

    fast = run()
    monkeypatch.setattr(_layers, "_fast", None)
    slow = run()
    assert len(fast) == len(slow)
    for a, c in zip(fast, slow):
        assert a.dtype == c.dtype and a.shape == c.shape and a.stride() == c.stride() and torch.equal(a, c)
