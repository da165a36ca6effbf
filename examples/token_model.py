"""A small language model of one block with experts, trained and then run token by token.

    python examples/token_model.py [--tokens T] [--vocabulary V] [--width H] [--hidden F]
                                   [--experts E] [--groups G] [--choices J] [--steps N]
                                   [--type bf16|f16|f32]

What lies around the block of expert_block.py in a language model: a norm before
it (`layer_norm`), the router's choice with a bias that keeps the experts' loads
even (`expert_choose`), a norm before the head, and the head's loss over the
vocabulary without its logits (`linear_cross_entropy`, whose weight is the
embedding).  torch looks the embeddings up and steps the optimiser.

Trains on a synthetic language (each token is followed by a fixed other one),
prints the loss, checks the trained model's losses one token at a time against
the batch, and exits non-zero if they differ.
"""
import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import dense_fp32_tiled_gb300 as sg
from examples.expert_block import Combine, ExpertLinear, Gather, Linear


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        stats = torch.empty((x.shape[0], 2), device=x.device)
        ctx.save_for_backward(x, weight, stats)
        return sg.layer_norm(x, weight, bias, stats=stats)

    @staticmethod
    def backward(ctx, dy):
        x, weight, stats = ctx.saved_tensors
        return sg.layer_norm_backward(dy.contiguous(), x, weight, stats)


class Choose(torch.autograd.Function):
    """(chosen, weights) of the router's logits; the bias decides with them and gets no gradient."""

    @staticmethod
    def forward(ctx, logits, choices, bias, groups, kept_groups):
        chosen, weights = sg.expert_choose(logits, choices, bias=bias, scoring="sigmoid", groups=groups, kept_groups=kept_groups,
                                           group_top=2)
        ctx.mark_non_differentiable(chosen)
        ctx.save_for_backward(logits, chosen)
        return chosen, weights

    @staticmethod
    def backward(ctx, _, dweights):
        logits, chosen = ctx.saved_tensors
        return sg.expert_choose_backward(dweights.contiguous(), logits, chosen, scoring="sigmoid"), None, None, None, None


class HeadLoss(torch.autograd.Function):
    """(loss, lse) of each token; weight is vocabulary x width."""

    @staticmethod
    def forward(ctx, x, weight, targets):
        loss, lse = sg.linear_cross_entropy(x, weight.t(), targets)
        ctx.save_for_backward(x, weight, targets, lse)
        return loss, lse

    @staticmethod
    def backward(ctx, dloss, dlse):
        x, weight, targets, lse = ctx.saved_tensors
        dx, dw = sg.linear_cross_entropy_backward(dloss.contiguous(), x, weight.t(), targets, lse, dlse=dlse.contiguous())
        return dx, dw.t(), None


class TokenModel(torch.nn.Module):
    def __init__(self, vocabulary, width, hidden, experts, groups, choices, dtype, device):
        super().__init__()
        self.experts, self.groups, self.choices = experts, groups, choices

        def weight(*shape, scale=None):
            return torch.nn.Parameter((torch.randn(shape, device=device) * (scale or 1 / math.sqrt(shape[-1]))).to(dtype))

        def vector(*shape, value=0.0):
            return torch.nn.Parameter(torch.full(shape, value, dtype=dtype, device=device))

        self.embedding = weight(vocabulary, width)
        self.norm1, self.norm1_bias = vector(width, value=1.0), vector(width)
        self.norm2, self.norm2_bias = vector(width, value=1.0), vector(width)
        self.router, self.router_bias = weight(experts, width), vector(experts)
        self.up, self.up_bias = weight(experts, hidden, width), vector(experts, hidden)
        self.down, self.down_bias = weight(experts, width, hidden), vector(experts, width)
        self.register_buffer("balance", torch.zeros(experts, device=device))

    def forward(self, tokens, targets):
        """(loss, lse, rows of each expert) of each token."""
        x = self.embedding[tokens]
        h = Norm.apply(x, self.norm1, self.norm1_bias)
        logits = Linear.apply(h, self.router, self.router_bias, "none")
        chosen, weights = Choose.apply(logits, self.choices, self.balance, self.groups, max(1, self.groups // 2))
        rows, offsets = sg.expert_sort(chosen, self.experts)
        xs = Gather.apply(h, rows, offsets)
        hidden = ExpertLinear.apply(xs, self.up, self.up_bias, offsets, "gelu_tanh")
        ys = ExpertLinear.apply(hidden, self.down, self.down_bias, offsets, "none")
        x = Combine.apply(ys, weights, x, rows, offsets)
        loss, lse = HeadLoss.apply(Norm.apply(x, self.norm2, self.norm2_bias), self.embedding, targets)
        return loss, lse, offsets[1:] - offsets[:-1]


def main() -> int:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--vocabulary", type=int, default=1000)
    ap.add_argument("--width", type=int, default=128)
    ap.add_argument("--hidden", type=int, default=256)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--groups", type=int, default=4)
    ap.add_argument("--choices", type=int, default=2)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--type", choices=["bf16", "f16", "f32"], default="f32")
    a = ap.parse_args()
    dtype = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[a.type]
    torch.manual_seed(0)
    model = TokenModel(a.vocabulary, a.width, a.hidden, a.experts, a.groups, a.choices, dtype, "cuda")
    following = torch.randperm(a.vocabulary, device="cuda")
    scale = 1024.0 if a.type == "f16" else 1.0  # of the loss: float16's gradients are small
    optimiser = torch.optim.Adam(model.parameters(), lr=1e-2 if a.type == "f32" else 3e-3, eps=1e-4)
    for step in range(a.steps):
        tokens = torch.randint(0, a.vocabulary, (a.tokens,), device="cuda")
        loss, lse, loads = model(tokens, following[tokens])
        loss = loss.mean() + 1e-4 * lse.square().mean()
        optimiser.zero_grad()
        (loss * scale).backward()
        optimiser.step()
        with torch.no_grad():  # experts asked for too often fall behind
            model.balance.add_(1e-3 * torch.sign(loads.float().mean() - loads.float()))
        if step % 10 == 0 or step + 1 == a.steps:
            print(f"step {step}: loss {float(loss.detach()):.4f}, fullest expert {int(loads.max())} of {int(loads.sum())} rows")
    with torch.no_grad():
        batch = model(tokens[:16], following[tokens[:16]])[0]
        single = torch.cat([model(tokens[i:i + 1], following[tokens[i:i + 1]])[0] for i in range(16)])
    off = float((batch - single).abs().max())
    print(f"16 tokens one at a time against the batch: losses differ by {off:.2e} at most")
    return 0 if off < (1e-4 if a.type == "f32" else 0.1) and sg.linear_timeouts() == 0 else 1


if __name__ == "__main__":
    sys.exit(main())
