"""expert_sort, expert_gather, expert_combine, expert_linear and their
gradients against the formulas in 64 bits (needs a GB300)."""
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


def _choices(seed, T, J, E, drop):
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, E, (T, J), generator=g)
    c[torch.rand((T, J), generator=g) < drop] = -1
    if T * J > 4:
        c.view(-1)[3] = E + 5  # dropped as well
    return c


def _sorted(choices, E):
    """rows and offsets, one choice at a time."""
    flat = choices.reshape(-1).tolist()
    counts = [0] * E
    for c in flat:
        if 0 <= c < E:
            counts[c] += 1
    offsets = [0]
    for n in counts:
        offsets.append(offsets[-1] + n)
    at, rows = offsets[:], []
    for c in flat:
        if 0 <= c < E:
            rows.append(at[c])
            at[c] += 1
        else:
            rows.append(-1)
    return torch.tensor(rows, dtype=torch.int32).reshape(choices.shape), torch.tensor(offsets, dtype=torch.int32)


@pytest.mark.parametrize("T,J,E,drop", [(1, 1, 1, 0), (1, 8, 64, 0), (7, 2, 3, 0.3), (33, 4, 16, 1.0), (1000, 6, 100, 0.1),
                                        (8192, 1, 8, 0), (20000, 2, 257, 0.05), (5000, 8, 1025, 0.01), (300, 64, 4096, 0),
                                        (9000, 2, 4096, 0.2)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(T, J, E, drop, dtype):
    c = _choices(T + E, T, J, E, drop)
    rows, offsets = sg.expert_sort(c.to(dtype).cuda(), E)
    want_rows, want_offsets = _sorted(c, E)
    assert torch.equal(offsets.cpu(), want_offsets)
    assert torch.equal(rows.cpu(), want_rows)


def test_sort_of_nothing():
    for T, J in ((0, 4), (5, 0)):
        rows, offsets = sg.expert_sort(torch.empty((T, J), dtype=torch.int32, device="cuda"), 6)
        assert rows.shape == (T, J) and (offsets == 0).all() and offsets.shape == (7,)


def test_sort_wide_integers():
    c = torch.tensor([[2 ** 32, 1], [-2 ** 33, 0]], dtype=torch.int64)  # dropped, not cut to 32 bits
    rows, offsets = sg.expert_sort(c.cuda(), 2)
    assert rows.tolist() == [[-1, 1], [-1, 0]] and offsets.tolist() == [0, 1, 2]


ROUTES = [(1, 1, 1, 1, 0), (1, 2, 4, 64, 0), (5, 3, 4, 7, 0.5), (4, 2, 3, 2048, 1.0), (100, 8, 32, 256, 0.1), (333, 6, 50, 129, 0.05),
          (64, 5, 9, 1000, 0.2), (3, 64, 80, 40, 0.1)]


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (3, 1)])
@pytest.mark.parametrize("T,J,E,H,drop", ROUTES)
def test_route_and_gradients(dtype, pad, offset, T, J, E, H, drop):
    dt = L.TYPES[dtype]
    g = L.rng(T + H)
    choices = _choices(T * 3 + H, T, J, E, drop).to(torch.int32).cuda()
    rows, offsets = sg.expert_sort(choices, E)
    x = L.strided(g, T, H, dt, pad, offset)
    out = torch.full((T * J, H + pad), 9.0, dtype=dt, device="cuda")
    xs = sg.expert_gather(x, rows, offsets, out=out[:, :H])
    want = torch.zeros(T * J, H, dtype=dt, device="cuda")
    for t in range(T):
        for j in range(J):
            if rows[t, j] >= 0:
                want[rows[t, j]] = x[t]
    assert torch.equal(xs, want) and (out[:, H:] == 9.0).all()
    # the places in no use hold NaN: nothing may read them
    ys = L.strided(g, T * J, H, dt, pad, offset)
    ys[int(offsets[E]):] = float("nan")
    weights = torch.rand((T, J), generator=g, device="cuda")
    weights[rows < 0] = float("nan")
    residual = L.strided(g, T, H, dt, pad, offset)
    kept = (rows >= 0)
    got_rows = torch.where(kept[..., None], ys[rows.clamp(min=0).long()].double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    wd = torch.where(kept, weights, torch.zeros_like(weights)).double()
    y = (got_rows * wd[..., None]).sum(1) + residual.double()
    S = (got_rows.abs() * wd[..., None]).sum(1) + residual.double().abs()
    L.assert_within(sg.expert_combine(ys, rows, weights, residual=residual), y, (J + 1) * 2.0 ** -24 * S + L.rounding(y, dt), "combine")
    y1, S1 = got_rows.sum(1), got_rows.abs().sum(1)
    L.assert_within(sg.expert_gather_backward(ys, rows), y1, J * 2.0 ** -24 * S1 + L.rounding(y1, dt), "gather backward")
    dy = L.strided(g, T, H, dt, pad, offset)
    dys, dweights = sg.expert_combine_backward(dy, ys, rows, weights, offsets)
    want_dys = torch.zeros(T * J, H, dtype=torch.float64, device="cuda")
    want_dys[rows[kept].long()] = (dy.double()[:, None, :] * wd[..., None])[kept]
    L.assert_within(dys, want_dys, L.rounding(want_dys, dt), "dys")
    dots = (got_rows * dy.double()[:, None, :]).sum(2)
    dot_s = (got_rows.abs() * dy.double().abs()[:, None, :]).sum(2)
    L.assert_within(dweights, dots, (H + 1) * 2.0 ** -24 * dot_s, "dweights")
    dys2, none = sg.expert_combine_backward(dy, ys, rows, weights, offsets, need_dweights=False)
    assert none is None and torch.equal(dys2, dys)


def test_combine_residual_in_place():
    g = L.rng(3)
    rows, offsets = sg.expert_sort(_choices(1, 20, 2, 4, 0.2).to(torch.int32).cuda(), 4)
    ys, r = L.randn(g, (40, 64), torch.bfloat16), L.randn(g, (20, 64), torch.bfloat16)
    want = sg.expert_combine(ys, rows, residual=r)
    assert torch.equal(sg.expert_combine(ys, rows, residual=r, out=r), want)


COUNTS = [[1], [0, 0, 0], [5, 0, 1, 200, 0, 63, 64, 65], [3] * 40, [1, 700], [130, 0, 129], [0, 0, 17]]
DIMS = [(64, 64), (130, 257), (8, 3), (640, 1024)]


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}e{sum(c)}r")
@pytest.mark.parametrize("tail", [0, 21])
def test_expert_linear(dtype, counts, tail):
    dt = L.TYPES[dtype]
    E, R = len(counts), sum(counts) + tail
    offsets = L.offsets_of(counts)
    at = offsets.tolist()
    for i, (N, K) in enumerate(DIMS):
        order, act = i % 2, L.ACTS[(i + E) % 5]
        g = L.rng(R + N)
        x = L.randn(g, (R, K), dt)
        if tail:
            x[at[-1]:] = float("nan")  # rows of no expert are not to matter
        w, b = L.weight(g, K, N, dt, order, (E,)), L.randn(g, (E, N), dt, 0.5)
        r = L.randn(g, (R, N), dt)
        z = torch.full((R, N), 5.0, dtype=dt, device="cuda")
        got = sg.expert_linear(x, w, offsets, bias=b, residual=r, activation=act, preact=z)
        for e in range(E):
            s = slice(at[e], at[e + 1])
            if at[e] == at[e + 1]:
                continue
            y, yb, zr, zb = L.forward_ref(x[s], w[e], b[e], r[s], act)
            L.assert_within(got[s], y, yb, f"expert {e} {N}x{K} {act}")
            L.assert_within(z[s], zr, zb, f"preact of expert {e} {N}x{K}")
        assert (got[at[-1]:] == 0).all() and (z[at[-1]:] == 0).all()


@pytest.mark.parametrize("dtype", L.TYPES)
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}e{sum(c)}r")
@pytest.mark.parametrize("tail", [0, 21])
def test_expert_linear_backward(dtype, counts, tail):
    dt = L.TYPES[dtype]
    E, R = len(counts), sum(counts) + tail
    offsets = L.offsets_of(counts)
    at = offsets.tolist()
    for i, (N, K) in enumerate(DIMS):
        order, act = (i + 1) % 2, L.ACTS[(i * 2 + E) % 5]
        g = L.rng(R * 2 + N)
        x, dy = L.randn(g, (R, K), dt), L.randn(g, (R, N), dt, 0.5)
        z = L.randn(g, (R, N), dt) if act != "none" else None
        if tail:
            x[at[-1]:] = float("nan")
            dy[at[-1]:] = float("nan")
        w = L.weight(g, K, N, dt, order, (E,))
        dx, dw, db = sg.expert_linear_backward(dy, x, w, offsets, preact=z, activation=act)
        assert (dx[at[-1]:] == 0).all()
        for e in range(E):
            s = slice(at[e], at[e + 1])
            if at[e] == at[e + 1]:
                assert (dw[e] == 0).all() and (db[e] == 0).all()
                continue
            refs = L.backward_ref(dy[s], x[s], w[e], z[s] if z is not None else None, act)
            for name, t, (ref, bound) in zip(("dx", "dw", "dbias"), (dx[s], dw[e], db[e]), refs):
                L.assert_within(t, ref, bound, f"{name} of expert {e} {N}x{K} {act}")


def test_expert_linear_neighbours_do_not_leak():
    # an expert's NaN rows stay in its own results, forward and in both gradients
    g = L.rng(4)
    counts = [70, 3, 100, 5]
    offsets = L.offsets_of(counts)
    at = offsets.tolist()
    x, dy, w = L.randn(g, (178, 96), torch.bfloat16), L.randn(g, (178, 80), torch.bfloat16), L.weight(g, 96, 80, torch.bfloat16, 1, (4,))
    clean = (sg.expert_linear(x, w, offsets), *sg.expert_linear_backward(dy, x, w, offsets))
    x2, dy2 = x.clone(), dy.clone()
    x2[at[1]:at[2]] = float("nan")
    dy2[at[1]:at[2]] = float("inf")
    got = (sg.expert_linear(x2, w, offsets), *sg.expert_linear_backward(dy2, x2, w, offsets))
    rows = [i for i in range(178) if not at[1] <= i < at[2]]
    for a, b in zip(got[:2], clean[:2]):
        assert torch.equal(a[rows], b[rows]) and not torch.isfinite(a[at[1]:at[2]]).any()
    for a, b in zip(got[2:], clean[2:]):
        assert torch.equal(a[[0, 2, 3]], b[[0, 2, 3]]) and not torch.isfinite(a[1]).any()


def test_whole_block_against_dense_experts():
    """Router to output and every gradient of a block of experts, against one product per expert in 64 bits."""
    g = L.rng(12)
    T, J, E, H, F = 60, 2, 5, 48, 72
    choices = torch.topk(torch.randn((T, E), generator=g, device="cuda"), J, dim=1).indices
    weights = torch.softmax(torch.randn((T, J), generator=g, device="cuda"), 1)
    x, w = L.randn(g, (T, H), torch.float32), L.weight(g, H, F, torch.float32, 1, (E,))
    rows, offsets = sg.expert_sort(choices, E)
    xs = sg.expert_gather(x, rows, offsets)
    z = torch.empty(T * J, F, device="cuda")
    ys = sg.expert_linear(xs, w, offsets, activation="silu", preact=z)
    y = sg.expert_combine(ys, rows, weights)
    dy = L.randn(g, (T, F), torch.float32)
    dys, dweights = sg.expert_combine_backward(dy, ys, rows, weights, offsets)
    dxs, dw, _ = sg.expert_linear_backward(dys, xs, w, offsets, preact=z, activation="silu", need_dbias=False)
    dx = sg.expert_gather_backward(dxs, rows)
    xd, wd, pd = (t.double().clone().requires_grad_() for t in (x, w, weights))
    all_e = torch.nn.functional.silu(torch.einsum("th,ehf->tef", xd, wd))
    ref = (all_e.gather(1, choices[..., None].expand(T, J, F)) * pd[..., None]).sum(1)
    ref.backward(dy.double())
    for got, want in ((y, ref.detach()), (dx, xd.grad), (dw, wd.grad), (dweights, pd.grad)):
        assert float((got.double() - want).norm() / want.norm()) < 1e-6
