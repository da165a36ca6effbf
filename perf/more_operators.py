"""The operators around a block with experts that are measured, and their plain forms.

The router's choice (`expert_choose`), the norm before a block (`layer_norm`), and the
loss of a language model's head without its logits (`linear_cross_entropy`), each with
its gradient.

`run(state)` makes one pass: in the plain form (elementary torch operations, in 32
bits, in 64 where values next to a border are compared, rounded once at the end), or,
with `own` set, through the package's calls.
"""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
PIECE = 16384  # of the vocabulary, in the plain forms
EPS = 1e-5


# ---- cases -------------------------------------------------------------------
# op          what is measured
# choose      each token's experts and weights from the router's logits
# choose_bwd  the gradient of the logits
# norm        y = layer norm of x; save: its rows' mean and 1 / deviation for training
# norm_bwd    dx, dweight, dbias
# loss        each token's -log softmax(x.w)[target], and its log sum of exponentials
# loss_bwd    dx, dw
#
# groups, kept, top: of `groups` groups of experts those `kept` with the largest sums
#     of their `top` best compete.  masked: share of tokens that are padding (all
#     logits -inf).
# wt: the weight is held as out x in, as checkpoints hold it, and handed over
#     transposed.  pad: elements between rows.  drop: share of tokens without a
#     target.  zloss: the loss has a term in the log sums too.  even: each token's
#     loss counts the same (a mean), else tokens have weights.


def listed():
    return [
        # a few decoded tokens pick their experts: latency
        {"name": "choose-decode", "op": "choose", "tokens": 8, "experts": 16, "choices": 2, "scoring": "softmax", "bias": False, "groups": 1, "kept": 1, "top": 1, "renorm": True, "scale": 1.0, "type": "bf16", "masked": 0.0},
        # a training batch over many experts in groups, balanced by a bias
        {"name": "choose-groups", "op": "choose", "tokens": 16384, "experts": 256, "choices": 8, "scoring": "sigmoid", "bias": True, "groups": 8, "kept": 4, "top": 2, "renorm": True, "scale": 2.5, "type": "f32", "masked": 0.0},
        # its gradient where every expert's score enters, some tokens padding
        {"name": "choose-grad", "op": "choose_bwd", "tokens": 16384, "experts": 100, "choices": 6, "scoring": "softmax", "renorm": False, "scale": 1.0, "type": "bf16", "masked": 0.05},
        # one token's norm before its block: latency
        {"name": "norm-token", "op": "norm", "m": 1, "n": 4096, "type": "bf16", "pad": 0, "save": False},
        # a long batch's norm, saved for training: bytes
        {"name": "norm", "op": "norm", "m": 16384, "n": 4096, "type": "bf16", "pad": 0, "save": True},
        # its gradient
        {"name": "norm-grad", "op": "norm_bwd", "m": 16384, "n": 4096, "type": "bf16", "pad": 0},
        # a gradient at the odd width of the repository's routing cases, in FP32
        {"name": "norm-grad-ragged", "op": "norm_bwd", "m": 5000, "n": 1001, "type": "f32", "pad": 0},
        # one token's likelihood: the head's weight is read once
        {"name": "loss-token", "op": "loss", "m": 1, "n": 32768, "k": 4096, "type": "bf16", "wt": True, "pad": 0, "drop": 0.0},
        # a training batch's loss
        {"name": "loss", "op": "loss", "m": 8192, "n": 65536, "k": 2048, "type": "bf16", "wt": True, "pad": 0, "drop": 0.02},
        # its gradient
        {"name": "loss-grad", "op": "loss_bwd", "m": 8192, "n": 65536, "k": 2048, "type": "bf16", "wt": True, "pad": 0, "drop": 0.02, "zloss": False, "even": True},
        # the sizes of the repository's ragged product, in FP32
        {"name": "loss-ragged-f32", "op": "loss", "m": 1000, "n": 1030, "k": 777, "type": "f32", "wt": False, "pad": 0, "drop": 0.1},
        # nothing is a multiple of anything, tokens with weights of their own, a term in the log sums
        {"name": "loss-grad-ragged", "op": "loss_bwd", "m": 1003, "n": 5003, "k": 641, "type": "f16", "wt": False, "pad": 0, "drop": 0.1, "zloss": True, "even": False},
    ]


def _log(rng, low, high):
    """A whole number between low and high, even over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A layer's width: as often a multiple of 64 as any number."""
    v = _log(rng, low, high)
    return max(64, v // 64 * 64) if rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(("choose", "choose", "choose_bwd", "norm", "norm_bwd", "loss", "loss_bwd"))
    c = {"op": op, "type": rng.choice(("bf16", "bf16", "f16", "f32"))}
    if op in ("choose", "choose_bwd"):
        e = _log(rng, 4, 256)
        c.update(tokens=_log(rng, 1, 16384), scoring=rng.choice(("softmax", "sigmoid")), renorm=rng.random() < 0.6, scale=rng.choice((1.0, 2.5)), masked=rng.choice((0.0, 0.0, 0.1)))
        groups, kept, top = 1, 1, 1
        if op == "choose":
            if rng.random() < 0.5:
                groups = rng.choice([g for g in (2, 3, 4, 8) if 2 * g <= e])
                e = e // groups * groups
                kept, top = rng.randint(1, groups), rng.choice((1, 2))
            c.update(bias=rng.random() < 0.5, groups=groups, kept=kept, top=top)
        # one choice's renormalised weight is a constant
        c.update(experts=e, choices=rng.randint(2 if op == "choose_bwd" and c["renorm"] else 1, min(8, e // groups * kept)))
    elif op in ("norm", "norm_bwd"):
        c.update(m=_log(rng, 1, 16384), n=_width(rng, 64, 16384), pad=rng.choice((0, 0, 8, 3)))
        while c["m"] * c["n"] > 16384 * 4096:
            c["m"] //= 2
        if op == "norm":
            c["save"] = rng.random() < 0.6
    else:
        c.update(m=_log(rng, 1, 8192), n=_width(rng, 64, 65536), k=_width(rng, 64, 2048), wt=rng.random() < 0.7, pad=rng.choice((0, 0, 8, 3)), drop=rng.choice((0.0, 0.02, 0.3)))
        if op == "loss_bwd":
            c.update(zloss=rng.random() < 0.3, even=rng.random() < 0.6)
    return c


# ---- inputs ------------------------------------------------------------------
def _rng(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEVICE) * scale).to(dtype)


def _in_rows(x, pad):
    """The same matrix with `pad` elements between its rows."""
    if not pad:
        return x
    wide = torch.zeros((x.shape[0], x.shape[1] + pad), dtype=x.dtype, device=x.device)
    wide[:, : x.shape[1]] = x
    return wide[:, : x.shape[1]]


def prepare(case, seed):
    c, g, dtype = dict(case), _rng(seed), TYPES[case["type"]]
    s = {"case": c}
    if c["op"] in ("choose", "choose_bwd"):
        t, e = c["tokens"], c["experts"]
        liked = torch.randn((e,), generator=g, device=DEVICE) * 0.5
        logits = torch.randn((t, e), generator=g, device=DEVICE) * 1.5 + liked
        if c["masked"]:
            logits = torch.where(torch.rand((t, 1), generator=g, device=DEVICE) < c["masked"], torch.full_like(logits, -math.inf), logits)
        s["logits"] = logits.to(dtype)
        if c["op"] == "choose":
            s["bias"] = torch.randn((e,), generator=g, device=DEVICE) * (0.05 if c["scoring"] == "sigmoid" else 0.3 / e) if c["bias"] else None
        else:
            s["dweights"] = torch.randn((t, c["choices"]), generator=g, device=DEVICE) * 0.1
            s["chosen"] = _choice(s["logits"], None, c["choices"], "softmax", 1, 1, 1)
    elif c["op"] in ("norm", "norm_bwd"):
        m, n, pad = c["m"], c["n"], c["pad"]
        # a residual stream: features of their own mean and size, a few far larger
        size = torch.exp(torch.randn((n,), generator=g, device=DEVICE) * 0.5)
        size = torch.where(torch.rand((n,), generator=g, device=DEVICE) < 0.002, size * 20, size)
        mean = torch.randn((n,), generator=g, device=DEVICE) * 0.5
        s["x"] = _in_rows((torch.randn((m, n), generator=g, device=DEVICE) * size + mean).to(dtype), pad)
        s["weight"] = (1 + torch.randn((n,), generator=g, device=DEVICE) * 0.2).to(dtype)
        if c["op"] == "norm":
            s["bias"] = _randn(g, (n,), dtype, 0.2)
        else:
            s["dy"] = _in_rows(_randn(g, (m, n), dtype, 0.1), pad)
            s["stats"] = _stats(s["x"].float())[0]
    else:
        m, n, k, pad = c["m"], c["n"], c["k"], c["pad"]
        w = torch.randn((n, k) if c["wt"] else (k, n), generator=g, device=DEVICE) * (2 / math.sqrt(k))
        w = w.to(dtype)
        s["w"] = w.t() if c["wt"] else w
        targets = torch.randint(0, n, (m,), generator=g, device=DEVICE)
        x = torch.randn((m, k), generator=g, device=DEVICE)
        # of half of the tokens the model knows something
        known = torch.rand((m, 1), generator=g, device=DEVICE) < 0.5
        x = torch.where(known, x + 3 * s["w"].t()[targets].float(), x)
        s["x"] = _in_rows(x.to(dtype), pad)
        if c["drop"]:
            targets = torch.where(torch.rand((m,), generator=g, device=DEVICE) < c["drop"], torch.full_like(targets, -100), targets)
        s["targets"] = targets
        if c["op"] == "loss_bwd":
            s["lse"] = _plain_loss(s)["lse"]
            count = (targets >= 0).sum().clamp(min=1)
            share = torch.ones((m,), device=DEVICE) if c["even"] else torch.rand((m,), generator=g, device=DEVICE) * 2
            s["dloss"] = share / count
            s["dlse"] = 2e-4 * s["lse"] / count if c["zloss"] else None
    return s


# ---- plain forms -------------------------------------------------------------
def _scores(l, scoring):
    if scoring == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _best(v):
    """The values of each row and their places in falling order, equal ones as they came."""
    return torch.sort(v, dim=1, descending=True, stable=True)


def _choice(logits, bias, choices, scoring, groups, kept, top):
    """tokens x choices experts, -1 where there are no more.  In 64 bits: scores next to one another decide."""
    l = logits.double()
    t, e = l.shape
    allowed = l > -math.inf
    s = _scores(l, scoring)
    v = s + bias.double() if bias is not None else s
    order = torch.where(allowed, v if bias is not None else l, torch.full_like(l, -math.inf))
    if groups > 1:
        size = e // groups
        inside = torch.where(allowed, v, torch.full_like(v, -math.inf)).reshape(t * groups, size)
        first = _best(inside)[0][:, : min(top, size)]
        total = torch.where(first > -math.inf, first, torch.zeros_like(first)).sum(1)
        total = torch.where(first[:, 0] > -math.inf, total, torch.full_like(total, -math.inf)).reshape(t, groups)
        if top == 1 and bias is None:
            total = order.reshape(t, groups, size).amax(2)
        keep = torch.zeros((t, groups), dtype=torch.bool, device=l.device).scatter_(1, _best(total)[1][:, :kept], True)
        order = torch.where(keep.repeat_interleave(size, dim=1), order, torch.full_like(order, -math.inf))
    value, at = _best(order)
    return torch.where(value[:, :choices] > -math.inf, at[:, :choices], torch.full_like(at[:, :choices], -1)).to(torch.int32)


def _plain_choose(s):
    c = s["case"]
    chosen = _choice(s["logits"], s["bias"], c["choices"], c["scoring"], c["groups"], c["kept"], c["top"])
    l, at = s["logits"].float(), chosen.clamp(min=0).long()
    weights = torch.where(chosen >= 0, torch.gather(_scores(l, c["scoring"]), 1, at), torch.zeros((), device=l.device))
    if c["renorm"]:
        weights = weights / torch.where(chosen[:, :1] >= 0, weights.sum(1, keepdim=True), torch.ones((), device=l.device))
    return {"chosen": chosen, "weights": weights * c["scale"]}


def _plain_choose_bwd(s):
    c, l, chosen = s["case"], s["logits"].float(), s["chosen"]
    none = torch.zeros((), device=l.device)
    at, some = chosen.clamp(min=0).long(), chosen >= 0
    p = _scores(l, c["scoring"])
    mine = torch.where(some, torch.gather(p, 1, at), none)
    dw = torch.where(some, s["dweights"] * c["scale"], none)
    if c["renorm"]:
        total = torch.where(some[:, :1], mine.sum(1, keepdim=True), torch.ones((), device=l.device))
        dw = (dw - (dw * mine).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(l).scatter_add_(1, at, torch.where(some, dw, none))
    if c["scoring"] == "sigmoid":
        dl = ds * p * (1 - p)
    else:
        dl = p * (ds - (ds * p).sum(1, keepdim=True))
    return {"dlogits": torch.where(some[:, :1], dl, none).to(s["logits"].dtype)}


def _stats(x):
    """Rows x 2: the mean, and 1 / deviation; and the rows without their mean."""
    n = x.shape[1]
    mean = x.sum(1, keepdim=True) / n
    d = x - mean
    rest = d.sum(1, keepdim=True) / n  # what the mean's rounding left
    d = d - rest
    return torch.cat([mean + rest, 1 / torch.sqrt((d * d).sum(1, keepdim=True) / n + EPS)], 1), d


def _plain_norm(s):
    dtype = s["x"].dtype
    stats, d = _stats(s["x"].float())
    y = (d * stats[:, 1:] * s["weight"].float() + s["bias"].float()).to(dtype)
    return {"y": y, "stats": stats} if s["case"]["save"] else {"y": y}


def _plain_norm_bwd(s):
    dtype, n = s["x"].dtype, s["case"]["n"]
    dy, rstd = s["dy"].float(), s["stats"][:, 1:]
    xhat = (s["x"].float() - s["stats"][:, :1]) * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - g.sum(1, keepdim=True) / n - xhat * ((g * xhat).sum(1, keepdim=True) / n))
    return {"dx": dx.to(dtype), "dweight": (dy * xhat).sum(0).to(dtype), "dbias": dy.sum(0).to(dtype)}


def _plain_loss(s):
    x, w, targets = s["x"].float(), s["w"], s["targets"]
    n = w.shape[1]
    high = torch.full((x.shape[0],), -math.inf, device=x.device)
    total, hit = torch.zeros_like(high), torch.zeros_like(high)
    for a in range(0, n, PIECE):
        z = x @ w[:, a : a + PIECE].float()
        higher = torch.maximum(high, z.amax(1))
        total = total * torch.exp(high - higher) + torch.exp(z - higher[:, None]).sum(1)
        high = higher
        at = targets - a
        inside = (at >= 0) & (at < z.shape[1])
        hit = torch.where(inside, torch.gather(z, 1, at.clamp(0, z.shape[1] - 1)[:, None])[:, 0], hit)
    lse = high + torch.log(total)
    return {"loss": torch.where((targets >= 0) & (targets < n), lse - hit, torch.zeros_like(lse)), "lse": lse}


def _plain_loss_bwd(s):
    dtype, x, w, targets = s["x"].dtype, s["x"].float(), s["w"], s["targets"]
    n = w.shape[1]
    g = torch.where((targets >= 0) & (targets < n), s["dloss"], torch.zeros_like(s["dloss"]))
    both = g + s["dlse"] if s["dlse"] is not None else g
    dx, dw = torch.zeros_like(x), []
    for a in range(0, n, PIECE):
        piece = w[:, a : a + PIECE].float()
        dz = torch.exp(x @ piece - s["lse"][:, None]) * both[:, None]
        at = targets - a
        inside = (at >= 0) & (at < dz.shape[1])
        dz.scatter_add_(1, at.clamp(0, dz.shape[1] - 1)[:, None], torch.where(inside, -g, torch.zeros_like(g))[:, None])
        dx += dz @ piece.t()
        dw.append((x.t() @ dz).to(dtype))
    return {"dx": dx.to(dtype), "dw": torch.cat(dw, 1)}


PLAIN = {"choose": _plain_choose, "choose_bwd": _plain_choose_bwd, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "loss": _plain_loss, "loss_bwd": _plain_loss_bwd}


# ---- the package's calls -----------------------------------------------------
def _own_choose(s):
    import dense_fp32_tiled_gb300 as sg
    c = s["case"]
    chosen, weights = sg.expert_choose(s["logits"], c["choices"], bias=s["bias"], scoring=c["scoring"], groups=c["groups"], kept_groups=c["kept"],
                                       group_top=c["top"], renormalize=c["renorm"], scale=c["scale"])
    return {"chosen": chosen, "weights": weights}


def _own_choose_bwd(s):
    import dense_fp32_tiled_gb300 as sg
    c = s["case"]
    return {"dlogits": sg.expert_choose_backward(s["dweights"], s["logits"], s["chosen"], scoring=c["scoring"], renormalize=c["renorm"], scale=c["scale"])}


def _own_norm(s):
    import dense_fp32_tiled_gb300 as sg
    c = s["case"]
    stats = torch.empty((c["m"], 2), device=s["x"].device) if c["save"] else None
    y = sg.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, stats=stats)
    return {"y": y, "stats": stats} if c["save"] else {"y": y}


def _own_norm_bwd(s):
    import dense_fp32_tiled_gb300 as sg
    dx, dweight, dbias = sg.layer_norm_backward(s["dy"], s["x"], s["weight"], s["stats"])
    return {"dx": dx, "dweight": dweight, "dbias": dbias}


def _own_loss(s):
    import dense_fp32_tiled_gb300 as sg
    loss, lse = sg.linear_cross_entropy(s["x"], s["w"], s["targets"])
    return {"loss": loss, "lse": lse}


def _own_loss_bwd(s):
    import dense_fp32_tiled_gb300 as sg
    dx, dw = sg.linear_cross_entropy_backward(s["dloss"], s["x"], s["w"], s["targets"], s["lse"], dlse=s["dlse"])
    return {"dx": dx, "dw": dw}


OWN = {"choose": _own_choose, "choose_bwd": _own_choose_bwd, "norm": _own_norm, "norm_bwd": _own_norm_bwd, "loss": _own_loss, "loss_bwd": _own_loss_bwd}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ---- what a pass cannot do without -------------------------------------------
def work(case):
    c, b = case, BYTES[case["type"]]
    if c["op"] == "choose":  # a comparison and a score per expert
        return {"bytes": c["tokens"] * (c["experts"] * b + 8 * c["choices"]) + (4 * c["experts"] if c["bias"] else 0), "flops": 5 * c["tokens"] * c["experts"]}
    if c["op"] == "choose_bwd":  # all logits where they all enter, else the chosen ones'
        read = c["experts"] if c["scoring"] == "softmax" and not c["renorm"] else c["choices"]
        return {"bytes": c["tokens"] * ((c["experts"] + read) * b + 8 * c["choices"]), "flops": 5 * c["tokens"] * read}
    if c["op"] == "norm":
        return {"bytes": b * (2 * c["m"] * c["n"] + 2 * c["n"]) + (8 * c["m"] if c["save"] else 0), "flops": 7 * c["m"] * c["n"]}
    if c["op"] == "norm_bwd":
        return {"bytes": b * (3 * c["m"] * c["n"] + 3 * c["n"]) + 8 * c["m"], "flops": 14 * c["m"] * c["n"]}
    m, n, k = c["m"], c["n"], c["k"]
    if c["op"] == "loss":
        return {"bytes": b * (m * k + k * n) + 16 * m, "flops": 2 * m * n * k}
    return {"bytes": 2 * b * (m * k + k * n) + (20 if c["zloss"] else 16) * m, "flops": 6 * m * n * k}


# ---- the definitions, in 64 bits -----------------------------------------------
def _exact_weights(l, chosen, c):
    """w (tokens x choices) with its graph back to l, from the definition."""
    s = torch.sigmoid(l) if c["scoring"] == "sigmoid" else torch.softmax(l, 1)
    some = chosen >= 0
    w = torch.gather(s, 1, chosen.clamp(min=0).long()).masked_fill(~some, 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).masked_fill(~some[:, :1], 1.0)
    return w * c["scale"]


def _exact_choice(l, bias, c):
    """One pick after another."""
    t, e = l.shape
    s = torch.sigmoid(l) if c["scoring"] == "sigmoid" else torch.softmax(l, 1)
    v = s if bias is None else s + bias
    lost = torch.isneginf(l)
    size = e // c["groups"]
    if c["groups"] > 1:
        left = v.masked_fill(lost, -math.inf).clone()
        total = torch.zeros((t, c["groups"]), dtype=torch.float64, device=l.device)
        for i in range(min(c["top"], size)):
            high, at = _first_max(left.view(t * c["groups"], size))
            total += high.view(t, -1) if i == 0 else high.view(t, -1).masked_fill(torch.isneginf(high.view(t, -1)), 0.0)
            left.view(t * c["groups"], size).scatter_(1, at[:, None], -math.inf)
        kept = torch.zeros_like(total, dtype=torch.bool)
        for _ in range(c["kept"]):
            _, at = _first_max(total.masked_fill(kept, -math.inf), kept)
            kept.scatter_(1, at[:, None], True)
        lost = lost | ~kept.repeat_interleave(size, 1)
    left = (l if bias is None else v).masked_fill(lost, -math.inf)
    picks = []
    for _ in range(c["choices"]):
        high, at = _first_max(left)
        picks.append(at.masked_fill(torch.isneginf(high), -1))
        left = left.scatter(1, at[:, None], -math.inf)
    return torch.stack(picks, 1).to(torch.int32)


def _first_max(v, taken=None):
    """Each row's maximum and the first place that has it (of those not taken)."""
    high = v.max(1).values
    place = torch.arange(v.shape[1], device=v.device).expand_as(v)
    there = v == high[:, None]
    if taken is not None:
        there = there & ~taken
    return high, place.masked_fill(~there, v.shape[1]).min(1).values.clamp(max=v.shape[1] - 1)


def exact(case, seed):
    s, op, c = prepare(case, seed), case["op"], case
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point() and k != "w"}
    if op == "choose":
        l = d["logits"]
        chosen = _exact_choice(l, d.get("bias"), c)
        return {"chosen": chosen, "weights": _exact_weights(l, chosen, c)}
    if op == "choose_bwd":
        l, chosen = d["logits"], s["chosen"]
        live = chosen[:, 0] >= 0
        dl = torch.zeros_like(l)
        if bool(live.any()):
            leaf = l[live].clone().requires_grad_()
            _exact_weights(leaf, chosen[live], c).backward(d["dweights"][live])
            dl[live] = leaf.grad
        return {"dlogits": dl}
    if op == "norm":
        var, mean = torch.var_mean(d["x"], 1, correction=0)
        rstd = torch.rsqrt(var + EPS)
        y = torch.addcmul(d["bias"], (d["x"] - mean[:, None]) * rstd[:, None], d["weight"])
        return {"y": y, "stats": torch.stack([mean, rstd], 1)} if c["save"] else {"y": y}
    if op == "norm_bwd":
        mean, rstd = d["stats"][:, 0], d["stats"][:, 1]
        h = torch.einsum("mn,m->mn", d["x"] - mean[:, None], rstd)
        g = torch.einsum("mn,n->mn", d["dy"], d["weight"])
        along = torch.einsum("mn,mn->m", g, h) / c["n"]
        dx = torch.einsum("m,mn->mn", rstd, g - g.mean(1)[:, None] - h * along[:, None])
        return {"dx": dx, "dweight": torch.einsum("mn,mn->n", d["dy"], h), "dbias": torch.einsum("mn->n", d["dy"])}
    # the loss: tokens some hundred at a time, the whole vocabulary at once
    w, t, n = s["w"].double(), s["targets"], c["n"]
    some = (t >= 0) & (t < n)
    step = max(1, 2 ** 27 // n)
    if op == "loss":
        loss, lse = [], []
        for a in range(0, c["m"], step):
            r = slice(a, a + step)
            z = d["x"][r] @ w
            lse.append(torch.logsumexp(z, 1))
            hit = z.gather(1, t[r].clamp(0, n - 1)[:, None])[:, 0]
            loss.append((lse[-1] - hit).masked_fill(~some[r], 0.0))
        return {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    g = d["dloss"].masked_fill(~some, 0.0)
    dw, dx = torch.zeros_like(w), []
    for a in range(0, c["m"], step):
        r = slice(a, a + step)
        dz = torch.exp(d["x"][r] @ w - d["lse"][r, None])
        dz *= (g[r] + (d["dlse"][r] if s["dlse"] is not None else 0.0))[:, None]
        rows = torch.nonzero(some[r])[:, 0]
        dz[rows, t[r][rows]] -= g[r][rows]
        dx.append(dz @ w.t())
        dw += d["x"][r].t() @ dz
    return {"dx": torch.cat(dx), "dw": dw}
