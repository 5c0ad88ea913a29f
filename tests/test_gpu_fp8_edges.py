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


def stack(n, rows, k, scale):
    ops = [R.integers(rows, k, 100 + e, "1d", scale) for e in range(n)]
    return fp4.fp8_stack([o for o, _ in ops]), [v for _, v in ops]


def offsets_of(counts):
    return torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("rows", [3, 400])
def test_every_row_dropped(rows, scale):
    x, _ = R.integers(rows, 300, 1, "1d", scale)
    w, _ = stack(5, 140, 300, scale)
    off = offsets_of([0] * 5)
    for dtype in (torch.bfloat16, torch.float32):
        assert (fp4.fp8_expert_gemm(x, w, off, dtype) == 0).all()
    for out in (torch.bfloat16, torch.float8_e4m3fn):
        h, gu = fp4.fp8_gated(x, w, "gelu", out, torch.bfloat16, off)
        assert (gu == 0).all()
        if out is torch.bfloat16:
            assert (h == 0).all()
        else:
            assert (h.q.view(torch.uint8) == 0).all() and (R.scale_values(h.s) == 1).all()


@pytest.mark.parametrize("n,counts,rows", [(1, [70], 90), (100, None, 300), (300, None, 900), (1024, None, 1500), (70, "hot", 200)])
def test_many_experts_and_one(n, counts, rows):
    """Exact on integers: more experts than a wave has lanes, one expert, one expert with nearly every row."""
    if counts is None:
        counts = [(7 * e) % 3 for e in range(n)]
    elif counts == "hot":
        counts = [1] * n
        counts[-2] = 100
    assert sum(counts) <= rows
    x, xv = R.integers(rows, 200, 3, "1d", "e8m0")
    w, wv = stack(n, 50, 200, "e8m0")
    y = fp4.fp8_expert_gemm(x, w, offsets_of(counts), torch.float32).cpu().double()
    at = 0
    for e, c in enumerate(counts):
        assert torch.equal(y[at:at + c], xv[at:at + c] @ wv[e].t()), e
        at += c
    assert (y[at:] == 0).all()


def test_no_rows_and_no_features():
    w, _ = stack(3, 64, 128, "e8m0")
    x, _ = R.integers(0, 128, 1, "1d", "e8m0")
    off = offsets_of([0, 0, 0])
    assert fp4.fp8_expert_gemm(x, w, off).shape == (0, 64)
    h, gu = fp4.fp8_gated(x, w, "silu", torch.float8_e4m3fn, torch.bfloat16, off)
    assert (h.rows, h.k) == (0, 32) and gu.shape == (0, 64)
    x, _ = R.integers(5, 128, 1, "1d", "e8m0")
    none, _ = R.integers(0, 128, 1, "1d", "e8m0")
    assert fp4.fp8_gemm(x, none).shape == (5, 0)
    h, gu = fp4.fp8_gated(x, none)
    assert h.shape == (5, 0) and gu is None
    h, _ = fp4.fp8_gated(x, none, out_dtype=torch.float8_e4m3fn)
    assert fp4.fp8_dequantize(h).shape == (5, 0)
    r, c = fp4.fp8_gated_grad(torch.zeros(0, 128, device="cuda"), torch.zeros(0, 256, device="cuda"))
    assert (r.rows, r.k, c.rows, c.k) == (0, 256, 256, 0)


def test_wrong_pairings_are_refused():
    x, _ = R.integers(5, 128, 1, "1d", "e8m0")
    w, _ = R.integers(6, 128, 2, "1d", "f32")
    with pytest.raises((ValueError, RuntimeError), match="scale type"):
        fp4.fp8_gemm(x, w)
    w, _ = R.integers(6, 256, 2, "1d", "e8m0")
    with pytest.raises((ValueError, RuntimeError), match="different k"):
        fp4.fp8_gemm(x, w)
    w, _ = R.integers(7, 128, 2, "1d", "e8m0")
    with pytest.raises(ValueError, match="stack gate and up"):
        fp4.fp8_gated(x, w)
    w, _ = R.integers(6, 128, 2, "1d", "e8m0")
    with pytest.raises(ValueError, match="plan"):
        fp4.fp8_gated(x, w, plan=offsets_of([5]))
    for out in (torch.empty(5, 7, device="cuda"), torch.empty(5, 6), torch.empty(6, 5, device="cuda").t()):
        with pytest.raises(ValueError):
            fp4.fp8_gemm(x, w, out=out)
