"""A mixture-of-experts feed-forward layer with FP4 expert weights: routing, forward and backward.

    python examples/moe_layer.py [--tokens 4096] [--hidden 4096] [--ffn 14336] [--experts 8] [--topk 2]

The expert weights are quantized once with 16x16 UE5M3 scales (TILE2D), which gives the forward and
the transposed operand of each; the layer keeps both as stacks. Activations stay bf16. The backward
pass gives the gradients of the input and of the router's weights (the FP4 weights are frozen).
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp4_block_scaled_tensor_amd as fp4  # noqa: E402


class MoELayer:
    """y[t] = sum_j w[t, j] * down_e(silu(up_e(x[t]))) over the experts e = ids[t, j] of token t."""

    def __init__(self, up: list[torch.Tensor], down: list[torch.Tensor]):
        """up: one [ffn, hidden] weight per expert, down: one [hidden, ffn] (bf16 or float32)."""
        def stacks(weights):
            pairs = [fp4.quantize(w, fp4.UE5M3, 16, fp4.TILE2D, amax=fp4.tensor_amax(w)) for w in weights]
            return fp4.stack_experts([p[0] for p in pairs]), fp4.stack_experts([p[1] for p in pairs])
        self.up, self.up_t = stacks(up)
        self.down, self.down_t = stacks(down)

    def forward(self, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor):
        """x [tokens, hidden], ids int [tokens, topk] (outside [0, experts): dropped), weights float32
        [tokens, topk] -> (y [tokens, hidden], what backward needs)."""
        plan = fp4.expert_sort(ids, self.up.n_experts)
        a = fp4.expert_linear(fp4.expert_gather(x, plan), self.up, plan)
        h = torch.nn.functional.silu(a.float()).to(a.dtype)
        ys = fp4.expert_linear(h, self.down, plan)
        return fp4.expert_combine(ys, weights, plan), (plan, a, ys, weights)

    def backward(self, dy: torch.Tensor, saved):
        """(dx [tokens, hidden], dweights [tokens, topk])."""
        plan, a, ys, weights = saved
        dys, dweights = fp4.expert_combine_grad(dy, ys, weights, plan)
        dh = fp4.expert_linear(dys, self.down_t, plan).float()
        s = torch.sigmoid(a.float())
        da = (dh * s * (1 + a.float() * (1 - s))).to(a.dtype)
        return fp4.expert_gather_grad(fp4.expert_linear(da, self.up_t, plan), plan), dweights


def route(logits: torch.Tensor, topk: int):
    """The topk experts of each token and their renormalised probabilities."""
    p, ids = torch.topk(torch.softmax(logits.float(), dim=1), topk, dim=1)
    return ids, (p / p.sum(dim=1, keepdim=True)).contiguous()


def main() -> None:
    p = argparse.ArgumentParser()
    for name, value in (("tokens", 4096), ("hidden", 4096), ("ffn", 14336), ("experts", 8), ("topk", 2)):
        p.add_argument("--" + name, type=int, default=value)
    c = p.parse_args()
    torch.manual_seed(0)
    rand = lambda *s: torch.randn(*s, device="cuda")   # noqa: E731
    layer = MoELayer([0.02 * rand(c.ffn, c.hidden) for _ in range(c.experts)],
                     [0.02 * rand(c.hidden, c.ffn) for _ in range(c.experts)])
    for tokens in (c.tokens, 1):   # a prompt, then a decode step
        x = rand(tokens, c.hidden).to(torch.bfloat16)
        ids, w = route(rand(tokens, c.experts), c.topk)
        dy = (1e-3 * rand(tokens, c.hidden)).to(torch.bfloat16)
        for _ in range(3):
            y, saved = layer.forward(x, ids, w)
            layer.backward(dy, saved)
        t = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
        t[0].record()
        y, saved = layer.forward(x, ids, w)
        t[1].record()
        layer.backward(dy, saved)
        t[2].record()
        torch.cuda.synchronize()
        print(f"{tokens} tokens: forward {t[0].elapsed_time(t[1]):.3f} ms, backward {t[1].elapsed_time(t[2]):.3f} ms, "
              f"|y| {y.float().norm().item():.4g}")


if __name__ == "__main__":
    main()
