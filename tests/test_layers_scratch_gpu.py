"""Scratch of the layer calls where calls do not follow one another: graphs
replayed on two streams at once, threads on one stream (needs a GB300)."""
import threading

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


def _inputs(seed, T=3000, H=200, F=264):
    g = L.rng(seed)
    return dict(x=L.randn(g, (T, H), torch.float32), w=L.weight(g, H, F, torch.float32, 1), dy=L.randn(g, (T, F), torch.float32),
                z=L.randn(g, (T, F), torch.float32), choices=torch.randint(0, 9, (T, 2), generator=g, device="cuda"))


def _run(i, stream=None):
    """Each kind of scratch: pieces of operands, dz and column sums, the sort's counts."""
    return (sg.linear(i["x"], i["w"], stream=stream),
            *sg.linear_backward(i["dy"], i["x"], i["w"], preact=i["z"], activation="silu", stream=stream),
            *sg.expert_sort(i["choices"], 9, stream=stream))


def test_two_graphs_at_once():
    inputs = [_inputs(1), _inputs(2)]
    want = [_run(i) for i in inputs]
    graphs, outs = [], []
    for i in inputs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):  # both on torch's one capture stream
            outs.append(_run(i))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(30):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    eager = [_run(i) for i in inputs]  # beside them, on the stream of the caller
    torch.cuda.synchronize()
    for got in (outs, eager):
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("given", [True, False])
def test_threads_on_one_stream(given):
    inputs = [_inputs(10 + k, T=400 + 100 * k) for k in range(4)]
    want = [_run(i) for i in inputs]
    stream = torch.cuda.Stream() if given else None
    torch.cuda.synchronize()
    start, got, errors = threading.Barrier(len(inputs)), [[] for _ in inputs], []

    def work(k):
        try:
            torch.cuda.set_device(0)
            start.wait()
            for _ in range(20):
                got[k].append(_run(inputs[k], stream))
        except Exception as e:  # reported below, on the main thread
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(inputs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for results, w in zip(got, want):
        for r in results:
            assert all(torch.equal(p, q) for p, q in zip(r, w))
