"""examples/fp8_ffn.py: it runs, and its gradients are those of the block up to the rounding of its operands."""
import os
import subprocess
import sys

import pytest
import torch

import fp4_block_scaled_tensor_amd as fp4

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.parametrize("scale", [fp4.F8_SCALE_E8M0, fp4.F8_SCALE_F32])
def test_gradients(scale):
    """E4M3 rounds a value by at most 2^-4 of it, 0.036 rms. At most six rounded tensors enter a result, and their
    errors are independent: 0.09 of its norm, and less than 0.15 with what bf16 and the least codes add."""
    from fp8_ffn import GatedFFN
    g = torch.Generator().manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g).cuda()   # noqa: E731
    tokens, hidden, f = 390, 512, 640
    up, down = hidden ** -0.5 * rand(2 * f, hidden), f ** -0.5 * rand(hidden, f)
    x, dy = rand(tokens, hidden).bfloat16(), rand(tokens, hidden).bfloat16()
    layer = GatedFFN(up, down, scale)
    y, saved = layer.forward(x)
    got = (y, *layer.backward(dy, saved))
    leaves = [t.double().requires_grad_() for t in (x, up, down)]
    gu = leaves[0] @ leaves[1].t()
    want_y = (torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]) @ leaves[2].t()
    want = (want_y.detach(), *torch.autograd.grad(want_y, leaves, dy.double()))
    for a, b in zip(got, want):
        assert (a.double() - b).norm() <= 0.15 * b.norm()


def test_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "fp8_ffn.py"), "--tokens", "300", "--hidden", "256",
                        "--ffn", "384"], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "forward" in r.stdout, r.stderr[-2000:]
