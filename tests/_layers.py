"""Helpers for the layer operators' tests: inputs, formulas in 64 bits, bounds.

Bounds, elementwise.  A K-term product in any order has an error of at most
K * 2**-23 * S for adds that may truncate, S = sum |x||w|; FP32 goes by
4 * (K + 8) * 2**-24 * S, the bound of the FP32 products (the 8: the pieces
left out, bias, activation and residual).  Rounding to the tensors' type adds
u |y|, u = 2**-8 for bfloat16 and 2**-11 for float16 (half a unit in the last
place, with 2**-25 below float16's normal range), FP32 2**-23.  The fast
exponential and quotient of the 16-bit types are within 2**-15 of the value.
No activation here has a slope above 1.2.
"""
import math

import torch

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {torch.float32: 2.0 ** -23, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def value(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def slope(z, act):
    """d value / d z, written out."""
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        h = torch.tanh(a * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + h) + 0.5 * z * (1 - h * h) * a * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def rounding(ref, dtype):
    return UNIT[dtype] * ref.abs() + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def product_bound(K, S, dtype):
    return 4 * (K + 8) * 2.0 ** -24 * S if dtype == torch.float32 else (K + 2) * 2.0 ** -23 * S


def act_bound(a, dtype):
    return (2.0 ** -21 if dtype == torch.float32 else 2.0 ** -15) * a.abs()


def assert_within(got, ref, bound, what):
    got = got.double().cpu()
    ref, bound = ref.cpu(), bound.cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN positions differ"
    err = (got - ref).abs()
    bad = ~(err <= bound) & ~torch.isnan(ref) & ~((got == ref) & torch.isinf(ref))
    if bad.any():
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, first at {i}: "
                             f"got {got[tuple(i)]}, want {ref[tuple(i)]}, bound {bound[tuple(i)]}")


def forward_ref(x, w, bias, residual, act):
    """(y, bound of y, z, bound of z) of act(x.w + bias) + residual for the tensors' type."""
    dtype = x.dtype
    xd, wd = x.double(), w.double()
    z = xd @ wd
    S = xd.abs() @ wd.abs()
    if bias is not None:
        z = z + bias.double()
        S = S + bias.double().abs()
    a = value(z, act)
    y = a if residual is None else a + residual.double()
    zb = product_bound(x.shape[1], S, dtype)
    yb = 1.2 * zb + act_bound(a, dtype) + rounding(y, dtype)
    if residual is not None:
        yb = yb + 2.0 ** -23 * (a.abs() + residual.double().abs())
    return y, yb, z, zb + rounding(z, dtype)


def backward_ref(dy, x, w, preact, act):
    """(dx, dw, dbias) and their bounds.  dz is rounded to the type before the two products
    (FP32: not), and its slope is within act_bound."""
    dtype = x.dtype
    g = dy.double()
    s = slope(preact.double(), act) if preact is not None else torch.ones_like(g)
    # the slopes are sums of terms of at most |s| + 1, each within act_bound
    gb = (act_bound(1 + s.abs(), dtype) * g.abs()) if preact is not None else torch.zeros_like(g)
    dz = g * s
    rb = gb + (rounding(dz, dtype) if dtype != torch.float32 and preact is not None else 0)
    xd, wd = x.double(), w.double()
    dx, dw, db = dz @ wd.t(), xd.t() @ dz, dz.sum(0)
    dxb = rb @ wd.abs().t() + product_bound(w.shape[1], (dz.abs() + rb) @ wd.abs().t(), dtype) + rounding(dx, dtype)
    dwb = xd.abs().t() @ rb + product_bound(x.shape[0], xd.abs().t() @ (dz.abs() + rb), dtype) + rounding(dw, dtype)
    dbb = gb.sum(0) + 2 * (x.shape[0] + 8) * 2.0 ** -24 * dz.abs().sum(0) + rounding(db, dtype)
    return (dx, dxb), (dw, dwb), (db, dbb)


def rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def strided(g, rows, cols, dtype, pad, offset=0, scale=1.0):
    """rows x cols inside a larger buffer of NaNs: row stride cols + pad, base `offset` elements off."""
    flat = torch.full((rows * (cols + pad) + offset + 8,), float("nan"), dtype=dtype, device="cuda")
    view = flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(randn(g, (rows, cols), dtype, scale))
    return view


def weight(g, K, N, dtype, order, lead=(), scale=None):
    s = scale if scale is not None else 1 / math.sqrt(max(K, 1))
    return randn(g, lead + (N, K), dtype, s).transpose(-1, -2) if order else randn(g, lead + (K, N), dtype, s)


def offsets_of(counts):
    return torch.tensor([0] + torch.tensor(counts, dtype=torch.int64).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
