"""The layer operators in captured graphs, on several streams at once, and with
many experts (needs a GB300)."""
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
    yield
    assert sg.linear_timeouts() == 0


def _inputs(seed, dt, T=200, J=2, E=6, H=96, F=136):
    g = L.rng(seed)
    return dict(x=L.randn(g, (T, H), dt), w=L.weight(g, H, F, dt, 1, (E,)), b=L.randn(g, (E, F), dt, 0.3),
                choices=torch.randint(0, E, (T, J), generator=g, device="cuda"),
                weights=torch.rand((T, J), generator=g, device="cuda"), dy=L.randn(g, (T, F), dt, 0.5),
                wd=L.weight(g, H, F, dt, 0), E=E)


def _block(i):
    """A block with experts and a dense layer, forward and backward: every operator."""
    rows, offsets = sg.expert_sort(i["choices"], i["E"])
    xs = sg.expert_gather(i["x"], rows, offsets)
    z = torch.empty((xs.shape[0], i["b"].shape[1]), dtype=xs.dtype, device="cuda")
    ys = sg.expert_linear(xs, i["w"], offsets, bias=i["b"], activation="silu", preact=z)
    zd = torch.empty((i["x"].shape[0], i["b"].shape[1]), dtype=xs.dtype, device="cuda")
    dense = sg.linear(i["x"], i["wd"], activation="gelu", preact=zd)
    y = sg.expert_combine(ys, rows, i["weights"], residual=dense)
    dys, dweights = sg.expert_combine_backward(i["dy"], ys, rows, i["weights"], offsets)
    dxs, dw, db = sg.expert_linear_backward(dys, xs, i["w"], offsets, preact=z, activation="silu")
    dx, dwd, dbd = sg.linear_backward(i["dy"], i["x"], i["wd"], preact=zd, activation="gelu")
    return y, dweights, dw, db, sg.expert_gather_backward(dxs, rows), dx, dwd, dbd


@pytest.mark.parametrize("dtype", L.TYPES)
def test_graph_of_a_block(dtype):
    i, other = _inputs(1, L.TYPES[dtype]), _inputs(2, L.TYPES[dtype])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _block(i)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = _block(i)
    for k, v in other.items():
        if isinstance(v, torch.Tensor):
            i[k].copy_(v)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for got, want in zip(out, _block(other)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", L.TYPES)
def test_streams_at_once(dtype):
    dt = L.TYPES[dtype]
    inputs = [_inputs(10 + k, dt, T=700 + 50 * k) for k in range(4)]
    want = [_block(i) for i in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    got = []
    for _ in range(5):
        got = []
        for i, s in zip(inputs, streams):
            with torch.cuda.stream(s):
                got.append(_block(i))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for p, q in zip(a, b):
            assert torch.equal(p, q)


def test_result_of_another_stream_waits_for_both_products():
    # what follows a backward pass in the stream comes after its second and its first product
    g = L.rng(5)
    x, dy, w = L.randn(g, (4096, 2048), torch.bfloat16), L.randn(g, (4096, 1024), torch.bfloat16), L.weight(g, 2048, 1024, torch.bfloat16, 1)
    dx, dw, db = sg.linear_backward(dy, x, w)
    torch.cuda.synchronize()
    for _ in range(20):
        a, b, c = sg.linear_backward(dy, x, w)
        sums = a.float().sum(), b.float().sum(), c.float().sum()  # queued at once, no synchronisation between
        assert torch.equal(sums[0], dx.float().sum()) and torch.equal(sums[1], dw.float().sum()) and torch.equal(sums[2], db.float().sum())


@pytest.mark.parametrize("E,R", [(300, 2000), (4096, 700)])
def test_many_experts(E, R):
    g = L.rng(E)
    mine = torch.sort(torch.randint(0, E, (R,), generator=g, device="cuda")).values
    counts = torch.bincount(mine, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    x, dy = L.randn(g, (R, 40), torch.bfloat16), L.randn(g, (R, 24), torch.bfloat16)
    w = L.weight(g, 40, 24, torch.bfloat16, 1, (E,))
    y = sg.expert_linear(x, w, offsets)
    dx, dw, db = sg.expert_linear_backward(dy, x, w, offsets)
    xd, wd, gd = x.double(), w.double()[mine], dy.double()
    S = torch.einsum("rk,rkn->rn", xd.abs(), wd.abs())
    ref = torch.einsum("rk,rkn->rn", xd, wd)
    L.assert_within(y, ref, L.product_bound(40, S, x.dtype) + L.rounding(ref, x.dtype), "y")
    ref, S = torch.einsum("rn,rkn->rk", gd, wd), torch.einsum("rn,rkn->rk", gd.abs(), wd.abs())
    L.assert_within(dx, ref, L.product_bound(24, S, x.dtype) + L.rounding(ref, x.dtype), "dx")
    outer = xd[:, :, None] * gd[:, None, :]
    ref = torch.zeros((E, 40, 24), dtype=torch.float64, device="cuda").index_add_(0, mine, outer)
    S = torch.zeros((E, 40, 24), dtype=torch.float64, device="cuda").index_add_(0, mine, outer.abs())
    L.assert_within(dw, ref, L.product_bound(int(counts.max()), S, x.dtype) + L.rounding(ref, x.dtype), "dw")
    ref = torch.zeros((E, 24), dtype=torch.float64, device="cuda").index_add_(0, mine, gd)
    S = torch.zeros((E, 24), dtype=torch.float64, device="cuda").index_add_(0, mine, gd.abs())
    L.assert_within(db, ref, 2 * (R + 8) * 2.0 ** -24 * S + L.rounding(ref, x.dtype), "dbias")


def test_offsets_out_of_order_stay_in_bounds():
    # wrong offsets give wrong rows, not wrong addresses: the buffers around the results stay as they were
    g = L.rng(7)
    x, dy, w = L.randn(g, (64, 32), torch.bfloat16), L.randn(g, (64, 48), torch.bfloat16), L.weight(g, 32, 48, torch.bfloat16, 1, (4,))
    for bad in ([0, 50, 20, 90, 64], [-5, -9, 3, 2 ** 30, 2 ** 31 - 1], [64, 0, 0, 0, 0], [10, 20, 30, 40, 50]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        guard = torch.full((3, 64, 48), 7.0, dtype=torch.bfloat16, device="cuda")
        sg.expert_linear(x, w, off, out=guard[1])
        sg.expert_linear_backward(dy, x, w, off)
        torch.cuda.synchronize()
        assert (guard[0] == 7).all() and (guard[2] == 7).all()
    rows = torch.tensor([[3, 900], [-7, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    guard = torch.full((3, 4, 32), 7.0, dtype=torch.bfloat16, device="cuda")
    sg.expert_gather(x[:2], rows, torch.tensor([0, 99], dtype=torch.int32, device="cuda"), out=guard[1])
    sg.expert_combine(x[:4], rows)
    torch.cuda.synchronize()
    assert (guard[0] == 7).all() and (guard[2] == 7).all()
