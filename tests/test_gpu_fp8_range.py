"""8-bit operators where an intermediate value could leave float32 though the result does not."""
import pytest
import torch

import fp4_block_scaled_tensor_amd as fp4
from tests import _fp8 as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gated_grad_of_the_largest_projections(dtype, act):
    """Slopes reach 1.13, so u times a slope may be past float32 where dh u act'(g) is far inside it. Tolerance: half
    a step of the output, and the arithmetic's 2^-20 of dh u (1 + |g|) and dh (1 + |g|) (sixteen float32 steps)."""
    big = torch.finfo(dtype).max
    g = torch.tensor([-3.0, -1.0, 0.5, 1.0, 1.4, 2.0, 2.4, 3.0, 5.0] * 2).to(dtype)
    u = torch.full((18,), big, dtype=dtype)
    u[9:] = -big
    dh = torch.tensor([1e-3, 2e-30, 0.75] * 6).to(dtype)
    gu = torch.cat([g, u])[None]
    got = fp4.gated_grad(dh[None].cuda(), gu.cuda(), act).cpu()
    g64, u64, d64 = g.double(), u.double(), dh.double()
    a, slope = R.act(g64, act)
    want = torch.cat([d64 * u64 * slope, d64 * a])
    mag = torch.cat([d64 * u64.abs() * (1 + g64.abs()), d64 * (1 + g64.abs())])
    assert ((got.double()[0] - want).abs() <= R.HALF[dtype] * want.abs() + 2.0 ** -20 * mag).all(), (got, want)


@pytest.mark.parametrize("scale", list(R.SCALES))
def test_fp8_gated_grad_of_the_largest_projections(scale):
    """The codes are those of the plain form's float32 result, none of them NaN."""
    g, u = R.randn(5, 128, 1, std=2.0), torch.full((5, 128), torch.finfo(torch.float32).max)
    dh, gu = R.randn(5, 128, 2, std=1e-3).cuda(), torch.cat([g, u], dim=1).cuda()
    d = fp4.gated_grad(dh, gu, "gelu")
    assert d.isfinite().all()
    r, c = fp4.fp8_gated_grad(dh, gu, "gelu", R.SCALES[scale])
    for t, v in ((r, d), (c, d.t().contiguous())):
        q, s = R.quantize_rows(v.cpu(), scale)
        assert torch.equal(t.q.cpu().view(torch.uint8), q)
        assert torch.equal(t.s.cpu() if scale == "f32" else t.s.cpu().view(torch.uint8), s)


@pytest.mark.parametrize("scale", list(R.SCALES))
def test_dequantize_of_a_long_transposed_operand(scale):
    """fp8_quantize's transposed view of more than 2^22 rows is an operand of more than 2^22 columns: too long for a
    product, not for its values."""
    rows = (1 << 22) + 200
    x = torch.randn(rows, 3, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda")
    t = fp4.fp8_quantize(x, fp4.COL, R.SCALES[scale])
    assert (t.rows, t.k) == (3, rows)
    v = fp4.fp8_dequantize(t)
    last = rows // 128 * 128
    for at in (slice(0, 256), slice(last - 256, rows)):   # whole blocks
        q, s = R.quantize_rows(x[at].t().contiguous().cpu(), scale)
        assert torch.equal(v[:, at].cpu(), R.values(q, s, "1d", 3, x[at].shape[0]).float())
    with pytest.raises(fp4.FP4Error, match="k must be at most"):
        fp4.fp8_gemm(t, t)
