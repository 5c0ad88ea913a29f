"""The example layer (sort, gather, experts' products, combine, and their gradients together) against the
same layer in float64 from the dequantized weights."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens,topk,dtype", [(1, 2, torch.float32), (9, 3, torch.float32), (300, 2, torch.float32),
                                               (64, 2, torch.bfloat16)])
def test_moe_layer_matches_float64(tokens, topk, dtype):
    import fp4_block_scaled_tensor_amd as fp4
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    hidden, ffn, experts = 128, 192, 5
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)   # noqa: E731
    layer = m.MoELayer([0.1 * rand(ffn, hidden) for _ in range(experts)], [0.1 * rand(hidden, ffn) for _ in range(experts)])

    def dense(stack):
        return [fp4.dequantize(fp4.QTensor(stack.q[e], stack.s[e], stack.g[e], stack.fmt, stack.block, stack.layout,
                                           stack.rows, stack.k)).double() for e in range(experts)]
    up, down = dense(layer.up), dense(layer.down)
    x = rand(tokens, hidden).to(dtype)
    ids, w = m.route(rand(tokens, experts), topk)
    if tokens > 1:
        ids[1, 0] = -1                               # a dropped slot
    y, saved = layer.forward(x, ids, w)
    dy = rand(tokens, hidden).to(dtype)
    dx, dw = layer.backward(dy, saved)

    x64 = x.double().requires_grad_(True)
    w64 = w.double().requires_grad_(True)
    y64 = []
    for t in range(tokens):
        row = torch.zeros(hidden, dtype=torch.float64, device="cuda")
        for j in range(topk):
            e = int(ids[t, j])
            if e >= 0:
                row = row + w64[t, j] * (down[e] @ torch.nn.functional.silu(up[e] @ x64[t]))
        y64.append(row)
    y64 = torch.stack(y64)
    (y64 * dy.double()).sum().backward()
    # The relative error of the norm. Each of at most four stored tensors on a path (gathered rows are copies)
    # rounds by half an ulp, 2^-8 (bf16) or 2^-24; the float32 sums of up to 192 products add 192 * 2^-23, and
    # silu and its derivative in float32 a few 2^-24. A factor of 2 for the amplification of a rounding in one
    # of the two factors of a product.
    lim = 2 * (4 * (2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24) + 4 * 192 * 2.0 ** -23)
    for got, want in ((y, y64), (dx, x64.grad), (dw, w64.grad)):
        err = (got.double() - want).norm() / want.norm()
        assert err <= lim, (err.item(), lim)
