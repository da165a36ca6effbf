"""A feed-forward block with experts, trained and then run token by token.

    python examples/expert_block.py [--tokens T] [--width H] [--hidden F]
                                    [--experts E] [--choices J] [--steps N]
                                    [--type bf16|f16|f32]

The block is the one of language models with experts: a router scores each token
(`linear`), its best J experts take it (`expert_sort`, `expert_gather`), each
expert is two products with an activation between them (`expert_linear`), and
their results join, weighted by the router, on top of the token itself
(`expert_combine` with its residual).  Every product, copy and sum, forward and
backward, is one of the package's operators; torch picks the experts (topk),
turns their scores into weights (softmax) and steps the optimiser.

Trains on a synthetic task (a fixed random block of the same shape), prints the
loss, checks the trained block's tokens one at a time against the batch, and
exits non-zero if the loss did not fall or the two differ.
"""
import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import dense_fp32_tiled_gb300 as sg


class Linear(torch.autograd.Function):
    """act(x.w + b); w is held as outputs x inputs."""

    @staticmethod
    def forward(ctx, x, weight, bias, activation):
        z = torch.empty((x.shape[0], weight.shape[0]), dtype=x.dtype, device=x.device) if activation != "none" else None
        y = sg.linear(x, weight.t(), bias, activation=activation, preact=z)
        ctx.save_for_backward(x, weight, z)
        ctx.activation = activation
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, z = ctx.saved_tensors
        dx, dw, db = sg.linear_backward(dy.contiguous(), x, weight.t(), preact=z, activation=ctx.activation)
        return dx, dw.t(), db, None


class ExpertLinear(torch.autograd.Function):
    """The same for rows sorted by expert; weight E x outputs x inputs, bias E x outputs."""

    @staticmethod
    def forward(ctx, x, weight, bias, offsets, activation):
        z = torch.empty((x.shape[0], weight.shape[1]), dtype=x.dtype, device=x.device) if activation != "none" else None
        y = sg.expert_linear(x, weight.transpose(1, 2), offsets, bias=bias, activation=activation, preact=z)
        ctx.save_for_backward(x, weight, offsets, z)
        ctx.activation = activation
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, offsets, z = ctx.saved_tensors
        dx, dw, db = sg.expert_linear_backward(dy.contiguous(), x, weight.transpose(1, 2), offsets, preact=z,
                                               activation=ctx.activation)
        return dx, dw.transpose(1, 2), db, None, None


class Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, rows, offsets):
        ctx.save_for_backward(rows)
        return sg.expert_gather(x, rows, offsets)

    @staticmethod
    def backward(ctx, dxs):
        return sg.expert_gather_backward(dxs.contiguous(), ctx.saved_tensors[0]), None, None


class Combine(torch.autograd.Function):
    """residual + the weighted sum of each token's rows."""

    @staticmethod
    def forward(ctx, ys, weights, residual, rows, offsets):
        ctx.save_for_backward(ys, weights, rows, offsets)
        return sg.expert_combine(ys, rows, weights, residual=residual)

    @staticmethod
    def backward(ctx, dy):
        ys, weights, rows, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        dys, dweights = sg.expert_combine_backward(dy, ys, rows, weights, offsets)
        return dys, dweights, dy, None, None


class ExpertBlock(torch.nn.Module):
    def __init__(self, width, hidden, experts, choices, dtype, device):
        super().__init__()
        self.experts, self.choices = experts, choices

        def weight(*shape):
            return torch.nn.Parameter((torch.randn(shape, device=device) / math.sqrt(shape[-1])).to(dtype))

        self.router = weight(experts, width)
        self.router_bias = torch.nn.Parameter(torch.zeros(experts, dtype=dtype, device=device))
        self.up, self.down = weight(experts, hidden, width), weight(experts, width, hidden)
        self.up_bias = torch.nn.Parameter(torch.zeros((experts, hidden), dtype=dtype, device=device))
        self.down_bias = torch.nn.Parameter(torch.zeros((experts, width), dtype=dtype, device=device))

    def forward(self, x):
        scores = Linear.apply(x, self.router, self.router_bias, "none")
        top, chosen = torch.topk(scores.float(), self.choices, dim=1)
        weights = torch.softmax(top, dim=1)
        rows, offsets = sg.expert_sort(chosen, self.experts)
        xs = Gather.apply(x, rows, offsets)
        h = ExpertLinear.apply(xs, self.up, self.up_bias, offsets, "silu")
        ys = ExpertLinear.apply(h, self.down, self.down_bias, offsets, "none")
        return Combine.apply(ys, weights, x, rows, offsets)


def main() -> int:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--choices", type=int, default=2)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--type", choices=["bf16", "f16", "f32"], default="f32")
    a = ap.parse_args()
    dtype = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[a.type]
    torch.manual_seed(0)
    shape = (a.width, a.hidden, a.experts, a.choices, dtype, "cuda")
    block, goal = ExpertBlock(*shape), ExpertBlock(*shape)
    optimiser = torch.optim.Adam(block.parameters(), lr=1e-2 if a.type == "f32" else 2e-3, eps=1e-4)
    losses = []
    for step in range(a.steps):
        x = torch.randn((a.tokens, a.width), device="cuda").to(dtype)
        with torch.no_grad():
            want = goal(x).float()
        loss = (block(x).float() - want).square().mean()
        optimiser.zero_grad()
        loss.backward()
        optimiser.step()
        losses.append(float(loss.detach()))
        if step % 10 == 0 or step + 1 == a.steps:
            print(f"step {step}: loss {losses[-1]:.4f}")
    with torch.no_grad():
        batch = block(x[:16]).float()
        single = torch.cat([block(x[i:i + 1]) for i in range(16)]).float()
    off = float((batch - single).norm() / batch.norm())
    print(f"16 tokens one at a time against the batch: relative difference {off:.2e}")
    fell = losses[-1] < 0.8 * losses[0]
    return 0 if fell and off < (1e-5 if a.type == "f32" else 2e-2) and sg.linear_timeouts() == 0 else 1


if __name__ == "__main__":
    sys.exit(main())
