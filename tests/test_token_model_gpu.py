"""A language model of one block with experts on the package's operators: runs,
and its gradients are the formula's (needs a GB300)."""
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


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_runs(dtype):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "token_model.py"), "--steps", "8", "--tokens", "300", "--type", dtype],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr


def _model(seed, dt, vocabulary=501, width=72, hidden=104, experts=12, groups=4, choices=3):
    from examples.token_model import TokenModel
    torch.manual_seed(seed)
    model = TokenModel(vocabulary, width, hidden, experts, groups, choices, dt, "cuda")
    with torch.no_grad():
        for n, p in model.named_parameters():
            if "bias" in n or "norm" in n:
                p.add_(torch.randn_like(p) * 0.1)
        model.balance.copy_(torch.randn(experts) * 0.02)
    return model


def _formula(model, tokens, targets, chosen):
    """The model in 64 bits with its choice of experts given."""
    p = {n: v.detach().double().requires_grad_() for n, v in model.named_parameters()}

    def norm(x, w, b):
        d = x - x.mean(1, keepdim=True)
        return d / torch.sqrt(d.square().mean(1, keepdim=True) + 1e-5) * w + b

    x = p["embedding"][tokens]
    h = norm(x, p["norm1"], p["norm1_bias"])
    s = torch.sigmoid(h @ p["router"].t() + p["router_bias"]).gather(1, chosen.long())
    w = s / s.sum(1, keepdim=True)
    up = torch.einsum("th,efh->tef", h, p["up"]) + p["up_bias"]
    act = 0.5 * up * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (up + 0.044715 * up ** 3)))
    ys = torch.einsum("tef,ehf->teh", act, p["down"]) + p["down_bias"]
    x = x + (ys.gather(1, chosen.long()[..., None].expand(-1, -1, ys.shape[2])) * w[..., None]).sum(1)
    z = norm(x, p["norm2"], p["norm2_bias"]) @ p["embedding"].t()
    lse = torch.logsumexp(z, 1)
    some = (targets >= 0) & (targets < z.shape[1])
    loss = torch.where(some, lse - z.gather(1, targets.clamp(0, z.shape[1] - 1)[:, None])[:, 0], torch.zeros_like(lse))
    return p, loss, lse


@pytest.mark.parametrize("tokens", [1, 37, 400])
def test_gradients(tokens):
    model = _model(1, torch.float32)
    g = L.rng(2)
    t = torch.randint(0, 501, (tokens,), generator=g, device="cuda")
    targets = torch.randint(0, 501, (tokens,), generator=g, device="cuda")
    if tokens > 30:
        targets[::7] = -100
    loss, lse, loads = model(t, targets)
    (loss.mean() + 1e-2 * lse.square().mean()).backward()
    with torch.no_grad():  # the same choice again
        h = sg.layer_norm(model.embedding[t], model.norm1, model.norm1_bias)
        chosen, _ = sg.expert_choose(sg.linear(h, model.router.t(), model.router_bias), 3, bias=model.balance, scoring="sigmoid", groups=4,
                                     kept_groups=2, group_top=2)
    p, want, want_lse = _formula(model, t, targets, chosen)
    (want.mean() + 1e-2 * want_lse.square().mean()).backward()
    # some hundred FP32 roundings one after the other, of which each is 2**-24 of the values it meets
    assert (loss - want).abs().max() < 1e-4 and (lse - want_lse).abs().max() < 1e-4
    for name, v in model.named_parameters():
        rel = float((v.grad.double() - p[name].grad).norm() / (p[name].grad.norm() + 1e-12))
        assert rel < 1e-4, (name, rel)


def _step(model, t, targets):
    model.zero_grad(set_to_none=True)
    loss, lse, loads = model(t, targets)
    (loss.mean() + 1e-2 * lse.square().mean()).backward()
    return [loss.detach(), lse.detach(), loads] + [p.grad for p in model.parameters()]


@pytest.mark.parametrize("dtype", L.TYPES)
def test_a_step_gives_the_same_bits_each_time(dtype):
    model = _model(3, L.TYPES[dtype])
    g = L.rng(4)
    t, targets = (torch.randint(0, 501, (333,), generator=g, device="cuda") for _ in range(2))
    with torch.no_grad():
        first = None
        for _ in range(4):
            h = sg.layer_norm(model.embedding[t], model.norm1, model.norm1_bias)
            logits = sg.linear(h, model.router.t(), model.router_bias)
            chosen, w = sg.expert_choose(logits, 3, bias=model.balance, scoring="sigmoid", groups=4, kept_groups=2, group_top=2)
            dlogits = sg.expert_choose_backward(w, logits, chosen, scoring="sigmoid")
            loss, lse = sg.linear_cross_entropy(h, model.embedding.t(), targets)
            dx, dw = sg.linear_cross_entropy_backward(loss, h, model.embedding.t(), targets, lse, dlse=lse)
            stats = torch.empty((333, 2), device="cuda")
            sg.layer_norm(h, model.norm1, stats=stats)
            now = [chosen, w, dlogits, loss, lse, dx, dw, *sg.layer_norm_backward(dx, h, model.norm1, stats)]
            assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
            first = now


@pytest.mark.parametrize("dtype", L.TYPES)
def test_a_captured_step(dtype):
    # forward and backward in a graph, beside an eager step of another model's leaves
    model, eager = _model(5, L.TYPES[dtype]), _model(6, L.TYPES[dtype])
    g = L.rng(7)
    t, targets, t2, targets2 = (torch.randint(0, 501, (130,), generator=g, device="cuda") for _ in range(4))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            _step(model, t, targets)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = _step(model, t, targets)
    torch.cuda.synchronize()
    t.copy_(t2)
    targets.copy_(targets2)
    for _ in range(3):
        graph.replay()
        _step(eager, t2, targets2)
    torch.cuda.synchronize()
    got = [o.clone() for o in out]
    # torch adds the embedding's gradient up with atomics: the first parameter's is not the same bits
    want = _step(model, t2, targets2)
    for i, (a, b) in enumerate(zip(got, want)):
        if i == 3:
            assert float((a.double() - b.double()).norm() / b.double().norm()) < 1e-2
        else:
            assert torch.equal(a, b), i


@pytest.mark.parametrize("dtype", L.TYPES)
def test_steps_on_several_streams_at_once(dtype):
    models = [_model(10 + i, L.TYPES[dtype]) for i in range(3)]
    g = L.rng(8)
    data = [tuple(torch.randint(0, 501, (200 + 40 * i,), generator=g, device="cuda") for _ in range(2)) for i in range(3)]
    want = [_step(m, *d) for m, d in zip(models, data)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in models]
    for _ in range(4):
        got = []
        for m, d, s in zip(models, data, streams):
            with torch.cuda.stream(s):
                got.append(_step(m, *d))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for i, (p, q) in enumerate(zip(a, b)):
                assert i == 3 or torch.equal(p, q), i
