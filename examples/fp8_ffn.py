"""A gated feed-forward block trained in 8 bits: forward, backward and the weights' gradients.

    python examples/fp8_ffn.py [--tokens 8192] [--hidden 4096] [--ffn 14336] [--scale e8m0]

Master weights are float32; a step quantizes them in 128 x 128 tiles (the forward and the transposed operand of
each), its input and its output's gradient in both views, and hands h from the gated product to the down
projection as codes. Only the gated projections (bf16) and the quantized input are kept for the backward pass.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp4_block_scaled_tensor_amd as fp4  # noqa: E402


class GatedFFN:
    """y = (silu(x . Wg^T) * (x . Wu^T)) . Wd^T with up = [Wg; Wu] [2 ffn, hidden] and down = Wd [hidden, ffn], float32.
    ffn is a multiple of 128."""

    def __init__(self, up: torch.Tensor, down: torch.Tensor, scale: int = fp4.F8_SCALE_E8M0):
        self.up, self.down, self.scale = up, down, scale

    def forward(self, x: torch.Tensor):
        """x [tokens, hidden] bf16 -> (y [tokens, hidden], what backward needs)."""
        up, up_t = fp4.fp8_quantize(self.up, fp4.TILE2D, self.scale)
        down, down_t = fp4.fp8_quantize(self.down, fp4.TILE2D, self.scale)
        rows, cols = fp4.fp8_quantize_rowcol(x, self.scale)
        h, gu = fp4.fp8_gated(rows, up, "silu", torch.float8_e4m3fn, save=torch.bfloat16)
        return fp4.fp8_gemm(h, down), (cols, gu, up_t, down_t)

    def backward(self, dy: torch.Tensor, saved):
        """dy [tokens, hidden] bf16 -> (dx bf16, d up float32, d down float32)."""
        cols, gu, up_t, down_t = saved
        dy_rows, dy_cols = fp4.fp8_quantize_rowcol(dy, self.scale)
        dh = fp4.fp8_gemm(dy_rows, down_t)
        d_rows, d_cols = fp4.fp8_gated_grad(dh, gu, "silu", self.scale)
        f = gu.shape[1] // 2
        h = (torch.nn.functional.silu(gu[:, :f].float()) * gu[:, f:].float()).to(gu.dtype)
        d_down = fp4.fp8_gemm(dy_cols, fp4.fp8_quantize(h, fp4.COL, self.scale), torch.float32)
        return fp4.fp8_gemm(d_rows, up_t), fp4.fp8_gemm(d_cols, cols, torch.float32), d_down


def main() -> None:
    p = argparse.ArgumentParser()
    for name, value in (("tokens", 8192), ("hidden", 4096), ("ffn", 14336)):
        p.add_argument("--" + name, type=int, default=value)
    p.add_argument("--scale", choices=("e8m0", "f32"), default="e8m0")
    c = p.parse_args()
    torch.manual_seed(0)
    rand = lambda *s: torch.randn(*s, device="cuda")   # noqa: E731
    layer = GatedFFN(c.hidden ** -0.5 * rand(2 * c.ffn, c.hidden), c.ffn ** -0.5 * rand(c.hidden, c.ffn),
                     fp4.F8_SCALE_E8M0 if c.scale == "e8m0" else fp4.F8_SCALE_F32)
    x, dy = rand(c.tokens, c.hidden).bfloat16(), (1e-3 * rand(c.tokens, c.hidden)).bfloat16()
    for _ in range(3):
        y, saved = layer.forward(x)
        layer.backward(dy, saved)
    t = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    t[0].record()
    y, saved = layer.forward(x)
    t[1].record()
    dx, d_up, d_down = layer.backward(dy, saved)
    t[2].record()
    torch.cuda.synchronize()
    print(f"{c.tokens} tokens: forward {t[0].elapsed_time(t[1]):.3f} ms, backward {t[1].elapsed_time(t[2]):.3f} ms, "
          f"|y| {y.float().norm().item():.4g}, |dx| {dx.float().norm().item():.4g}, |d up| {d_up.norm().item():.4g}")


if __name__ == "__main__":
    main()
