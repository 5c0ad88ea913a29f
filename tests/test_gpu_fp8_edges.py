"""8-bit operators at the ends of their ranges: gates of any size, infinite scales, a gradient written over its input."""
import math

import pytest
import torch

import fp4_block_scaled_tensor_amd as fp4
from tests import _fp8 as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated_grad_of_any_finite_gate(act):
    """Slopes of 1 and 0 far from zero, also where a square or a cube of the gate is infinite. Tolerance: the
    activations' own, 1e-5 of a value or 1e-6."""
    big = torch.tensor([30.0, 1e5, 1e13, 1e20, 3e38])
    g = torch.cat([big, -big, torch.zeros(1)])
    n = g.numel()
    dh, gu = torch.ones(1, n), torch.cat([g, torch.ones(n)])[None]
    got = fp4.gated_grad(dh.cuda(), gu.cuda(), act).cpu().double()[0]
    y, slope = R.act(g.double(), act)
    want = torch.cat([slope, y])
    assert ((got - want).abs() <= 1e-5 * want.abs() + 1e-6).all(), (got, want)


def test_gated_grad_of_a_closed_gate_is_zero():
    """A slope of 0 times dh u past the type's range."""
    for act, gate in (("silu", -3e38), ("gelu", -60.0), ("gelu_tanh", -60.0)):
        dh, gu = torch.full((1, 9), 1e30), torch.cat([torch.full((1, 9), gate), torch.full((1, 9), 1e30)], dim=1)
        assert (fp4.gated_grad(dh.cuda(), gu.cuda(), act) == 0).all(), act


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,f", [(1, 8), (33, 1001), (40, 4096)])
def test_gated_grad_over_its_input(rows, f, dtype):
    dh, gu = R.randn(rows, f, 1, dtype).cuda(), R.randn(rows, 2 * f, 2, dtype).cuda()
    want = fp4.gated_grad(dh, gu, "gelu")
    got = fp4.gated_grad(dh, gu, "gelu", out=gu)
    assert got is gu and torch.equal(got, want)


def ones(rows, k, s):
    q = torch.zeros(rows, R.blocks(k) * R.B)
    q[:, :k] = 1.0
    return fp4.F8Tensor(q.to(R.F8).cuda(), s.cuda(), fp4.FP4_SCALES_1D, rows, k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("blocks", [1, 9, 33])
@pytest.mark.parametrize("m", [1, 40])
def test_infinite_scale_of_the_last_block(m, blocks, dtype):
    k = 128 * blocks
    s = torch.ones(m, blocks)
    s[0, -1] = math.inf
    y = fp4.fp8_gemm(ones(m, k, s), ones(70, k, torch.ones(70, blocks)), dtype).cpu()
    assert (y[0] == math.inf).all() and (y[1:] == k).all()


@pytest.mark.parametrize("m", [1, 40])
def test_sums_past_the_range(m):
    for dtype in (torch.bfloat16, torch.float32):
        a, b = torch.full((m, 9), 127 + 100, dtype=torch.uint8), torch.full((70, 9), 127 + 60, dtype=torch.uint8)
        y = fp4.fp8_gemm(ones(m, 9 * 128, a), ones(70, 9 * 128, b), dtype)
        assert (y == math.inf).all()
