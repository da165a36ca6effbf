"""expert_choose, layer_norm and linear_cross_entropy: through the extension and
the interpreter, on a given stream, with rows apart and far apart (needs a GB300)."""
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_tiled_gb300 as sg
from dense_fp32_tiled_gb300 import _layers
from tests import _layers as L
from tests.test_choose_gpu import check as check_choice
from tests.test_cross_entropy_gpu import check_backward, check_forward, inputs
from tests.test_norm_gpu import check_backward as check_norm_backward
from tests.test_norm_gpu import check_forward as check_norm_forward

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


def _inputs(dt, seed=1):
    g = L.rng(seed)
    x, w, t = inputs(g, 70, 333, 48, dt, 1)
    return dict(x=x, w=w, t=t, weight=L.randn(g, (48,), dt), logits=L.randn(g, (70, 24), dt), bias=torch.randn((24,), generator=g, device="cuda") * 0.1,
                dloss=torch.randn((70,), generator=g, device="cuda"), dw=torch.randn((70, 4), generator=g, device="cuda"))


def _run(i, **kw):
    """Every call once."""
    stats = torch.empty((70, 2), device="cuda")
    y = sg.layer_norm(i["x"], i["weight"], i["weight"], eps=1e-4, stats=stats, **kw)
    chosen, w = sg.expert_choose(i["logits"], 4, bias=i["bias"], scoring="sigmoid", groups=4, kept_groups=2, group_top=2, scale=1.5, **kw)
    loss, lse = sg.linear_cross_entropy(i["x"], i["w"], i["t"], **kw)
    return [y, stats, chosen, w, loss, lse, *sg.layer_norm_backward(y, i["x"], i["weight"], stats, **kw),
            sg.expert_choose_backward(i["dw"], i["logits"], chosen, scoring="sigmoid", scale=1.5, **kw),
            *sg.linear_cross_entropy_backward(i["dloss"], i["x"], i["w"], i["t"], lse, dlse=loss, **kw)]


@pytest.mark.parametrize("dtype", L.TYPES)
def test_both_ways_agree(monkeypatch, dtype):
    _layers._load()
    i = _inputs(L.TYPES[dtype])
    fast = _run(i)
    monkeypatch.setattr(_layers, "_fast", None)
    for a, b in zip(fast, _run(i)):
        assert a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride() and torch.equal(a, b)


def test_on_a_given_stream():
    i = _inputs(torch.bfloat16)
    want = _run(i)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = _run(i, stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_numbers_of_other_kinds():
    # whole numbers where others are meant, NumPy's and torch's: served by the interpreter's way
    i = _inputs(torch.float32)
    assert torch.equal(sg.layer_norm(i["x"], eps=1), sg.layer_norm(i["x"], eps=1.0))
    for a, b in zip(sg.expert_choose(i["logits"], torch.tensor(3).item(), scale=2), sg.expert_choose(i["logits"], 3, scale=2.0)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", L.TYPES)
def test_what_lies_between_rows_stays(dtype):
    dt = L.TYPES[dtype]
    g = L.rng(3)
    lib, kind = _layers._load(), {"f32": 0, "bf16": 1, "f16": 2}[dtype]
    M, N, K, E = 37, 130, 52, 20

    def room(rows, cols):
        whole = torch.full((rows + 2, cols + 5), 7.0, dtype=dt, device="cuda")
        return whole, whole[1:rows + 1, 2:cols + 2]

    def untouched(whole, inside):
        before = torch.full_like(whole, 7.0)
        before[1:inside.shape[0] + 1, 2:inside.shape[1] + 2] = inside
        return torch.equal(whole, before) and not (inside == 7.0).all()

    x, w, t = inputs(g, M, N, K, dt, 0)
    whole, y = room(M, K)
    sg.layer_norm(x, out=y)
    assert untouched(whole, y)
    stats = torch.empty((M, 2), device="cuda")
    sg.layer_norm(x, stats=stats)
    stream = torch.cuda.current_stream().cuda_stream
    whole, dx = room(M, K)
    assert lib.layer_norm_backward(kind, M, K, x.data_ptr(), x.stride(0), x.data_ptr(), x.stride(0), None, stats.data_ptr(), dx.data_ptr(),
                                   dx.stride(0), None, None, None, 0, stream) == 0
    assert untouched(whole, dx)
    logits = L.randn(g, (M, E), dt)
    chosen, weights = sg.expert_choose(logits, 3)
    whole, dl = room(M, E)
    assert lib.expert_choose_backward(kind, M, E, 3, weights.data_ptr(), chosen.data_ptr(), logits.data_ptr(), E, 0, 1, 1.0, dl.data_ptr(),
                                      dl.stride(0), stream) == 0
    assert untouched(whole, dl) and torch.equal(dl, sg.expert_choose_backward(weights, logits, chosen))
    loss, lse = sg.linear_cross_entropy(x, w, t)
    want = sg.linear_cross_entropy_backward(loss, x, w, t, lse)
    whole, dx = room(M, K)
    whole_w, dw = room(K, N)
    need = lib.linear_cross_entropy_backward_workspace_size(kind, M, N, K, x.data_ptr(), x.stride(0), w.data_ptr(), w.stride(0), 0, 1, 1)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda").fill_(0xff)
    assert lib.linear_cross_entropy_backward(kind, M, N, K, loss.data_ptr(), None, x.data_ptr(), x.stride(0), w.data_ptr(), w.stride(0), 0, t.data_ptr(),
                                             8, lse.data_ptr(), dx.data_ptr(), dx.stride(0), dw.data_ptr(), dw.stride(0), ws.data_ptr(), need, stream) == 0
    assert untouched(whole, dx) and untouched(whole_w, dw)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1]) and (ws[need:] == 0xff).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_far_apart(dtype):
    # offsets past 2**31 elements
    dt = L.TYPES[dtype]
    g = L.rng(4)
    far = 2 ** 30 + 8
    flat = torch.zeros(2 * far + 4096, dtype=dt, device="cuda")
    x = flat.as_strided((3, 1000), (far, 1))
    x.copy_(L.randn(g, (3, 1000), dt))
    check_norm_forward(x, L.randn(g, (1000,), dt), None, 1e-5)
    check_norm_backward(x, x, L.randn(g, (1000,), dt))
    check_choice(x, 8)
    out = torch.zeros(2 * far + 4096, dtype=dt, device="cuda").as_strided((3, 1000), (far, 1))
    check_norm_forward(x, None, None, 1e-5, out=out)
    w = L.weight(g, 1000, 300, dt, 1)
    t = torch.tensor([5, 299, 17], device="cuda")
    loss, lse, z, zb = check_forward(x, w, t)
    check_backward(x, w, t, lse, z, zb, torch.ones(3, device="cuda"))
    wide = flat.as_strided((3, 1000), (far, 1)).t()  # and a weight of three columns far apart
    loss, lse, z, zb = check_forward(L.randn(g, (5, 1000), dt), wide, torch.tensor([0, 1, 2, -1, 2], device="cuda"))


def test_a_weight_of_more_than_2_to_the_31_values():
    g = L.rng(5)
    M, N, K = 20, 140001, 15400
    w = torch.randn((N, K), generator=g, device="cuda", dtype=torch.bfloat16).mul_(2 / K ** 0.5)
    x = L.randn(g, (M, K), torch.bfloat16)
    t = torch.randint(N - 50, N, (M,), generator=g, device="cuda")
    loss, lse = sg.linear_cross_entropy(x, w.t(), t)
    z = torch.cat([x.double() @ w[a:a + 20000].double().t() for a in range(0, N, 20000)], 1)
    want = torch.logsumexp(z, 1)
    assert (lse - want).abs().max() < 1e-4 and (loss - (want - z.gather(1, t[:, None])[:, 0])).abs().max() < 1e-4
    dx, dw = sg.linear_cross_entropy_backward(torch.ones(M, device="cuda"), x, w.t(), t, lse)
    dz = torch.exp(z - want[:, None])
    dz[torch.arange(M, device="cuda"), t] -= 1
    part = slice(N - 2000, N)
    ref = dz[:, part].t() @ x.double()
    got = dw.t()[part].double()
    assert float((got - ref).norm() / ref.norm()) < 5e-3
    ref = sum(dz[:, a:a + 20000] @ w[a:a + 20000].double() for a in range(0, N, 20000))
    assert float((dx.double() - ref).norm() / ref.norm()) < 5e-3
