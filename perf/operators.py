"""The operators of a feed-forward layer that are measured, and their plain forms.

A dense layer's product with bias, activation and residual (`linear`), its gradient
(`linear_backward`), the same product over rows sorted by expert (`expert_linear`,
`expert_linear_backward`), and the way of the tokens to their experts and back
(`expert_sort`, `expert_gather`, `expert_combine` and their gradients).

`run(state)` makes one pass: in the plain form (elementary torch operations, in 32
bits, rounded once at the end), or, with `own` set, through the package's calls.
"""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ---- cases -------------------------------------------------------------------
# op          what is measured
# linear      y = act(x.w + bias) + residual
# linear_bwd  dx, dw, dbias from dy, x, w and the saved argument of the activation
# expert      y[r] = act(x[r].w[e] + bias[e]) for the rows r of expert e
# expert_bwd  its dx, dw, dbias
# route       sort the tokens by expert, copy them into that order, and join what
#             the experts made of them, each weighted by its router
# route_bwd   the gradients of the two copies and of the weights
#
# wt: the weight is held as out x in, as checkpoints hold it, and handed over
#     transposed.  pad: elements between the rows of the activations.


def listed():
    return [
        # one token through a projection: latency, and the weight's bytes
        {"name": "token", "op": "linear", "m": 1, "n": 4096, "k": 4096, "type": "bf16", "act": "silu", "wt": True, "pad": 0, "save": False},
        # the sizes of the repository's ragged product: nothing is a multiple of anything
        {"name": "ragged-f32", "op": "linear", "m": 1000, "n": 1030, "k": 777, "type": "f32", "act": "gelu", "wt": False, "pad": 0, "save": True},
        # the repository's headline product as a layer in FP32
        {"name": "square-f32", "op": "linear", "m": 4096, "n": 4096, "k": 4096, "type": "f32", "act": "silu", "wt": False, "pad": 0, "save": False},
        # a prompt through the wide half of a feed-forward block, its argument saved for training
        {"name": "prompt", "op": "linear", "m": 8192, "n": 8192, "k": 4096, "type": "bf16", "act": "gelu_tanh", "wt": True, "pad": 0, "save": True},
        # a small layer's gradient in FP32
        {"name": "grad-f32", "op": "linear_bwd", "m": 1024, "n": 1024, "k": 1024, "type": "f32", "act": "gelu", "wt": False, "pad": 0},
        # a training step's gradient
        {"name": "grad", "op": "linear_bwd", "m": 8192, "n": 8192, "k": 2048, "type": "bf16", "act": "silu", "wt": True, "pad": 0},
        # a batch of decoded tokens over many experts: a few rows each, every weight read once
        {"name": "experts-decode", "op": "expert", "rows": 128, "experts": 64, "n": 1024, "k": 2048, "type": "bf16", "act": "silu", "wt": True, "tail": 0},
        # a training batch's gradient through the experts
        {"name": "experts-grad", "op": "expert_bwd", "rows": 16384, "experts": 16, "n": 4096, "k": 2048, "type": "bf16", "act": "silu", "wt": True, "tail": 0},
        # few rows, odd sizes, rows that no expert got
        {"name": "experts-grad-ragged", "op": "expert_bwd", "rows": 1500, "experts": 9, "n": 1000, "k": 641, "type": "f16", "act": "gelu", "wt": False, "tail": 37},
        # a few decoded tokens on their way to the experts and back: latency
        {"name": "route-decode", "op": "route", "tokens": 8, "choices": 2, "experts": 16, "h": 2048, "type": "bf16", "drop": 0.0},
        # a long batch's way there and back: bytes
        {"name": "route", "op": "route", "tokens": 16384, "choices": 4, "experts": 64, "h": 4096, "type": "bf16", "drop": 0.01},
        # its gradient, at an odd width in FP32, with dropped choices
        {"name": "route-grad", "op": "route_bwd", "tokens": 5000, "choices": 6, "experts": 100, "h": 1001, "type": "f32", "drop": 0.05},
    ]


def _log(rng, low, high):
    """A whole number between low and high, even over the logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    v = min(high, max(low, v))
    return v + 1 if v == 3072 else v


def _width(rng, low, high):
    """A layer's width: as often a multiple of 64 as any number."""
    v = _log(rng, low, high)
    if rng.random() < 0.5:
        v = max(64, v // 64 * 64)
        v = v + 64 if v == 3072 else v
    return v


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_bwd", "expert", "expert_bwd", "route", "route_bwd"))
    c = {"op": op, "type": rng.choice(("bf16", "bf16", "f16", "f32"))}
    if op in ("linear", "linear_bwd"):
        c.update(m=_log(rng, 1, 8192), n=_width(rng, 64, 8192), k=_width(rng, 64, 4096), act=rng.choice(ACTIVATIONS), wt=rng.random() < 0.6, pad=rng.choice((0, 0, 8, 3)))
        if op == "linear":
            c["save"] = rng.random() < 0.4
    elif op in ("expert", "expert_bwd"):
        e = _log(rng, 2, 64)
        c.update(rows=_log(rng, 2, 16384), experts=e, n=_width(rng, 64, 4096 if e <= 16 else 1024), k=_width(rng, 64, 2048), act=rng.choice(ACTIVATIONS), wt=rng.random() < 0.6)
        c["tail"] = rng.choice((0, 0, c["rows"] // 40))
    else:
        e = _log(rng, 4, 256)
        c.update(tokens=_log(rng, 1, 16384), choices=rng.randint(1, min(8, e)), experts=e, h=_width(rng, 64, 4096), drop=rng.choice((0.0, 0.02, 0.2)))
        while c["tokens"] * c["choices"] * c["h"] > 65536 * 4096:
            c["tokens"] //= 2
    return c


# ---- inputs ------------------------------------------------------------------
def _rng(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEVICE) * scale).to(dtype)


def _rows(g, m, width, dtype, pad, scale=1.0):
    return _randn(g, (m, width + pad), dtype, scale)[:, :width]


def _weight(g, k, n, dtype, wt, lead=()):
    """k x n, as n x k in memory where `wt`; spread so that a product keeps its rows' size."""
    if wt:
        return _randn(g, lead + (n, k), dtype, 1 / math.sqrt(k)).transpose(-1, -2)
    return _randn(g, lead + (k, n), dtype, 1 / math.sqrt(k))


def _choices(g, tokens, choices, experts, drop):
    """Each token's experts by a router's scores, some experts asked for more than others, and the weights that it gives them."""
    liked = torch.randn((experts,), generator=g, device=DEVICE) * 0.5
    scores = torch.randn((tokens, experts), generator=g, device=DEVICE) + liked
    top, at = torch.topk(scores, choices, dim=1)
    weights = torch.softmax(top, dim=1)
    if drop:
        at = torch.where(torch.rand(at.shape, generator=g, device=DEVICE) < drop, torch.full_like(at, -1), at)
    return at.to(torch.int32), weights


def prepare(case, seed):
    c, g, dtype = dict(case), _rng(seed), TYPES[case["type"]]
    s = {"case": c}
    if c["op"] in ("linear", "linear_bwd"):
        m, n, k, pad = c["m"], c["n"], c["k"], c["pad"]
        s["x"] = _rows(g, m, k, dtype, pad)
        s["w"] = _weight(g, k, n, dtype, c["wt"])
        if c["op"] == "linear":
            s["bias"] = _randn(g, (n,), dtype, 0.5)
            s["residual"] = _rows(g, m, n, dtype, pad)
        else:
            s["dy"] = _rows(g, m, n, dtype, pad, 0.1)
            s["z"] = _rows(g, m, n, dtype, pad) if c["act"] != "none" else None
    elif c["op"] in ("expert", "expert_bwd"):
        r, e, n, k = c["rows"], c["experts"], c["n"], c["k"]
        share = torch.softmax(torch.randn((e,), generator=g, device=DEVICE) * 0.5, 0)
        mine = torch.multinomial(share, r - c["tail"], replacement=True, generator=g)
        counts = torch.bincount(mine, minlength=e)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["most"] = int(counts.max())  # the fullest expert's rows: what a padded batch is sized by
        s["x"] = _randn(g, (r, k), dtype)
        s["w"] = _weight(g, k, n, dtype, c["wt"], (e,))
        if c["op"] == "expert":
            s["bias"] = _randn(g, (e, n), dtype, 0.5)
        else:
            s["dy"] = _randn(g, (r, n), dtype, 0.1)
            s["z"] = _randn(g, (r, n), dtype) if c["act"] != "none" else None
    else:
        t, j, e, h = c["tokens"], c["choices"], c["experts"], c["h"]
        s["experts"], s["weights"] = _choices(g, t, j, e, c["drop"])
        if c["op"] == "route":
            s["x"] = _randn(g, (t, h), dtype)
            s["ys"] = _randn(g, (t * j, h), dtype)
            s["residual"] = _randn(g, (t, h), dtype)
        else:
            s["dy"] = _randn(g, (t, h), dtype, 0.1)
            s["ys"] = _randn(g, (t * j, h), dtype)
            s["dxs"] = _randn(g, (t * j, h), dtype, 0.1)
            s["rows"], s["offsets"] = _order(s["experts"], e)
    return s


# ---- plain forms -------------------------------------------------------------
def _act(z, name):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        h = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + h) + 0.5 * z * (1 - h * h) * a * (1 + 3 * 0.044715 * z * z)
    return None


def _order(experts, e):
    """Where each choice's row goes (-1: nowhere), and where each expert's rows begin."""
    flat = experts.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < e), flat, torch.full_like(flat, e))
    by = torch.argsort(key, stable=True)
    at = torch.empty_like(by)
    at[by] = torch.arange(by.numel(), device=by.device)
    rows = torch.where(key < e, at, torch.full_like(at, -1)).reshape(experts.shape)
    counts = torch.zeros(e + 1, dtype=torch.long, device=by.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([counts.new_zeros(1), counts[:e].cumsum(0)])
    return rows.to(torch.int32), offsets.to(torch.int32)


def _places(offsets, rows, e, most):
    """Each row's place in a batch of e times `most` rows; the rows of no expert share the place after the last."""
    r = torch.arange(rows, device=offsets.device)
    ends = offsets[1:].long()
    mine = torch.bucketize(r, ends, right=True)
    begins = torch.cat([offsets[:-1].long(), ends[-1:]])
    place = mine * most + r - begins[mine]
    return torch.where(mine < e, place, torch.full_like(place, e * most)), mine


def _batched(x, place, e, most):
    b = x.new_zeros((e * most + 1, x.shape[1]))
    b[place] = x
    b[e * most] = 0
    return b[: e * most].reshape(e, most, x.shape[1])


def _unbatched(b, place):
    flat = b.reshape(-1, b.shape[-1])
    return torch.cat([flat, flat.new_zeros((1, flat.shape[1]))])[place]


def _plain_linear(s):
    c, dtype = s["case"], s["x"].dtype
    z = s["x"].float() @ s["w"].float() + s["bias"].float()
    y = _act(z, c["act"]) + s["residual"].float()
    return {"y": y.to(dtype), "z": z.to(dtype)} if c["save"] else {"y": y.to(dtype)}


def _plain_linear_bwd(s):
    c, dtype = s["case"], s["x"].dtype
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_slope(s["z"].float(), c["act"])
    dx, dw = dz @ s["w"].float().t(), s["x"].float().t() @ dz
    return {"dx": dx.to(dtype), "dw": dw.to(dtype), "dbias": dz.sum(0).to(dtype)}


def _plain_expert(s):
    c, dtype, e, most = s["case"], s["x"].dtype, s["case"]["experts"], s["most"]
    place, _ = _places(s["offsets"], c["rows"], e, most)
    z = torch.bmm(_batched(s["x"].float(), place, e, most), s["w"].float()) + s["bias"].float()[:, None, :]
    return {"y": _unbatched(_act(z, c["act"]), place).to(dtype)}


def _plain_expert_bwd(s):
    c, dtype, e, most = s["case"], s["x"].dtype, s["case"]["experts"], s["most"]
    place, _ = _places(s["offsets"], c["rows"], e, most)
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_slope(s["z"].float(), c["act"])
    dz = _batched(dz, place, e, most)
    dx = _unbatched(torch.bmm(dz, s["w"].float().transpose(1, 2)), place)
    dw = torch.bmm(_batched(s["x"].float(), place, e, most).transpose(1, 2), dz)
    return {"dx": dx.to(dtype), "dw": dw.to(dtype), "dbias": dz.sum(1).to(dtype)}


def _picked(ys, rows):
    """tokens x choices x h: each choice's row, zeros where it was dropped."""
    got = ys.float()[rows.clamp(min=0).long()]
    return torch.where((rows >= 0)[..., None], got, got.new_zeros(()))


def _plain_route(s):
    c, dtype = s["case"], s["x"].dtype
    rows, offsets = _order(s["experts"], c["experts"])
    n = rows.numel()
    at = torch.where(rows >= 0, rows, torch.full_like(rows, n)).reshape(-1).long()
    xs = s["x"].new_zeros((n + 1, c["h"]))
    xs[at] = s["x"].repeat_interleave(c["choices"], dim=0)
    xs[n] = 0
    y = (_picked(s["ys"], rows) * s["weights"][..., None]).sum(1) + s["residual"].float()
    return {"rows": rows, "offsets": offsets, "xs": xs[:n], "y": y.to(dtype)}


def _plain_route_bwd(s):
    c, dtype, rows = s["case"], s["dy"].dtype, s["rows"]
    n = rows.numel()
    dy = s["dy"].float()
    dweights = (_picked(s["ys"], rows) * dy[:, None, :]).sum(2)
    at = torch.where(rows >= 0, rows, torch.full_like(rows, n)).reshape(-1).long()
    dys = dy.new_zeros((n + 1, c["h"]))
    dys[at] = (dy[:, None, :] * s["weights"][..., None]).reshape(n, c["h"])
    dys[n] = 0
    return {"dys": dys[:n].to(dtype), "dweights": dweights, "dx": _picked(s["dxs"], rows).sum(1).to(dtype)}


PLAIN = {"linear": _plain_linear, "linear_bwd": _plain_linear_bwd, "expert": _plain_expert, "expert_bwd": _plain_expert_bwd, "route": _plain_route, "route_bwd": _plain_route_bwd}


# ---- the package's calls -----------------------------------------------------
def _own_linear(s):
    import dense_fp32_tiled_gb300 as sg
    c = s["case"]
    z = torch.empty((c["m"], c["n"]), dtype=s["x"].dtype, device=s["x"].device) if c["save"] else None
    y = sg.linear(s["x"], s["w"], bias=s["bias"], residual=s["residual"], activation=c["act"], preact=z)
    return {"y": y, "z": z} if c["save"] else {"y": y}


def _own_linear_bwd(s):
    import dense_fp32_tiled_gb300 as sg
    dx, dw, dbias = sg.linear_backward(s["dy"], s["x"], s["w"], preact=s["z"], activation=s["case"]["act"])
    return {"dx": dx, "dw": dw, "dbias": dbias}


def _own_expert(s):
    import dense_fp32_tiled_gb300 as sg
    return {"y": sg.expert_linear(s["x"], s["w"], s["offsets"], bias=s["bias"], activation=s["case"]["act"])}


def _own_expert_bwd(s):
    import dense_fp32_tiled_gb300 as sg
    dx, dw, dbias = sg.expert_linear_backward(s["dy"], s["x"], s["w"], s["offsets"], preact=s["z"], activation=s["case"]["act"])
    return {"dx": dx, "dw": dw, "dbias": dbias}


def _own_route(s):
    import dense_fp32_tiled_gb300 as sg
    rows, offsets = sg.expert_sort(s["experts"], s["case"]["experts"])
    xs = sg.expert_gather(s["x"], rows, offsets)
    y = sg.expert_combine(s["ys"], rows, s["weights"], residual=s["residual"])
    return {"rows": rows, "offsets": offsets, "xs": xs, "y": y}


def _own_route_bwd(s):
    import dense_fp32_tiled_gb300 as sg
    dys, dweights = sg.expert_combine_backward(s["dy"], s["ys"], s["rows"], s["weights"], s["offsets"])
    dx = sg.expert_gather_backward(s["dxs"], s["rows"])
    return {"dys": dys, "dweights": dweights, "dx": dx}


OWN = {"linear": _own_linear, "linear_bwd": _own_linear_bwd, "expert": _own_expert, "expert_bwd": _own_expert_bwd, "route": _own_route, "route_bwd": _own_route_bwd}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ---- what a pass cannot do without -------------------------------------------
def work(case):
    c, b = case, BYTES[case["type"]]
    saved = c.get("act") != "none"
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": b * (m * k + k * n + n + m * n * (3 if c["save"] else 2)), "flops": 2 * m * n * k}
    if c["op"] == "linear_bwd":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": b * (m * n * (2 if saved else 1) + 2 * m * k + 2 * k * n + n), "flops": 4 * m * n * k}
    if c["op"] in ("expert", "expert_bwd"):
        r, n, k = c["rows"] - c["tail"], c["n"], c["k"]
        met = min(c["experts"], r)  # experts with rows, at most: the others' weights are not read
        if c["op"] == "expert":
            return {"bytes": b * (r * k + met * (k * n + n) + c["rows"] * n) + 4 * c["experts"], "flops": 2 * r * n * k}
        return {"bytes": b * (r * n * (2 if saved else 1) + r * k + c["rows"] * k + met * k * n + c["experts"] * (k * n + n)) + 4 * c["experts"], "flops": 4 * r * n * k}
    t, j, h = c["tokens"], c["choices"], c["h"]
    if c["op"] == "route":  # choices and weights; x, residual and y; xs written and ys read
        return {"bytes": 3 * 4 * t * j + b * (3 * t * h + 2 * t * j * h), "flops": 2 * t * j * h}
    return {"bytes": 3 * 4 * t * j + b * (2 * t * h + 3 * t * j * h), "flops": 4 * t * j * h}


# ---- the definitions, in 64 bits -----------------------------------------------
def _phi(z):
    return torch.special.ndtr(z)


def _value_and_slope(z, name):
    """The activation and its derivative at z, in 64 bits."""
    if name == "relu":
        return z.relu(), torch.heaviside(z, z.new_zeros(()))
    if name == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * torch.sigmoid(-z)
    if name == "gelu":
        return z * _phi(z), _phi(z) + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":  # 0.5 (1 + tanh u) = sigmoid(2 u)
        r = math.sqrt(8 / math.pi)
        p = torch.sigmoid(r * (z + 0.044715 * z ** 3))
        return z * p, p + z * p * (1 - p) * r * (1 + 0.134145 * z.square())
    return z, torch.ones_like(z)


def exact(case, seed):
    s, op, act = prepare(case, seed), case["op"], case.get("act")
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if op == "linear":
        z = torch.addmm(d["bias"], d["x"], d["w"])
        y = _value_and_slope(z, act)[0] + d["residual"]
        return {"y": y, "z": z} if case["save"] else {"y": y}
    if op == "linear_bwd":
        dz = d["dy"] if s["z"] is None else d["dy"] * _value_and_slope(d["z"], act)[1]
        return {"dx": torch.einsum("mn,kn->mk", dz, d["w"]), "dw": torch.einsum("mk,mn->kn", d["x"], dz), "dbias": torch.einsum("mn->n", dz)}
    if op in ("expert", "expert_bwd"):
        at, rows = s["offsets"].tolist(), case["rows"]
        if op == "expert":
            y = torch.zeros((rows, case["n"]), dtype=torch.float64, device=DEVICE)
            for e in range(case["experts"]):
                r = slice(at[e], at[e + 1])
                y[r] = _value_and_slope(d["x"][r] @ d["w"][e] + d["bias"][e], act)[0]
            return {"y": y}
        dz = d["dy"] if s["z"] is None else d["dy"] * _value_and_slope(d["z"], act)[1]
        dx = torch.zeros_like(d["x"])
        dw, dbias = torch.zeros(d["w"].shape, dtype=torch.float64, device=DEVICE), []
        for e in range(case["experts"]):
            r = slice(at[e], at[e + 1])
            dx[r] = dz[r] @ d["w"][e].t()
            dw[e] = d["x"][r].t() @ dz[r]
            dbias.append(dz[r].sum(0))
        return {"dx": dx, "dw": dw, "dbias": torch.stack(dbias)}
    # the routes: one choice at a time
    t, j, e, h = case["tokens"], case["choices"], case["experts"], case["h"]
    if op == "route":
        asked = s["experts"].cpu().reshape(-1).tolist()
        rows, offsets = [-1] * len(asked), [0]
        held = [[] for _ in range(e)]
        for i, a in enumerate(asked):
            if 0 <= a < e:
                held[a].append(i)
        for mine in held:
            for q, i in enumerate(mine):
                rows[i] = offsets[-1] + q
            offsets.append(offsets[-1] + len(mine))
        rows = torch.tensor(rows, dtype=torch.int32, device=DEVICE).reshape(t, j)
        xs = torch.zeros((t * j, h), dtype=torch.float64, device=DEVICE)
        y = d["residual"].clone()
        for q in range(j):
            at = rows[:, q].long()
            kept = torch.nonzero(at >= 0).reshape(-1)
            xs.index_copy_(0, at[kept], d["x"][kept])
            y.index_add_(0, kept, d["ys"][at[kept]] * d["weights"][kept, q, None])
        return {"rows": rows, "offsets": torch.tensor(offsets, dtype=torch.int32, device=DEVICE), "xs": xs, "y": y}
    dys = torch.zeros((t * j, h), dtype=torch.float64, device=DEVICE)
    dx = torch.zeros((t, h), dtype=torch.float64, device=DEVICE)
    dweights = torch.zeros((t, j), dtype=torch.float64, device=DEVICE)
    for q in range(j):
        at = s["rows"][:, q].long()
        kept = torch.nonzero(at >= 0).reshape(-1)
        dys.index_copy_(0, at[kept], d["dy"][kept] * d["weights"][kept, q, None])
        dx.index_add_(0, kept, d["dxs"][at[kept]])
        dweights[kept, q] = torch.einsum("th,th->t", d["ys"][at[kept]], d["dy"][kept])
    return {"dys": dys, "dweights": dweights, "dx": dx}
