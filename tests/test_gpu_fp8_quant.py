"""fp8_quantize in every view, its decode, and the gated gradient, bit for bit or against float64."""
import pytest
import torch

import fp4_block_scaled_tensor_amd as fp4
from tests import _fp8 as R

pytestmark = pytest.mark.gpu
SIZES = [(1, 1), (1, 128), (5, 200), (128, 128), (129, 257), (200, 1000), (300, 77), (2, 4096)]


def inputs(rows, cols, dtype, seed=0):
    """Heavy-tailed rows over many magnitudes, with zero blocks, exact powers of two and values at the scale's edge."""
    x = R.randn(rows, cols, seed) * torch.pow(2.0, R.randn(rows, cols, seed + 1) * 6)
    if rows > 3:
        x[3] = 0
        x[1] = torch.pow(2.0, torch.randint(-20, 20, (cols,), generator=torch.Generator().manual_seed(seed)).float())
        x[2] = 448.0
        x[2, ::3] = -449.0
    return x.to(dtype)


def same(t, q, s, rows, k):
    assert (t.rows, t.k) == (rows, k)
    assert torch.equal(t.q.cpu().view(torch.uint8), q)
    got = t.s.cpu() if t.s.dtype == torch.float32 else t.s.cpu().view(torch.uint8)
    assert torch.equal(got, s)


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_views(rows, cols, dtype, scale):
    x = inputs(rows, cols, dtype)
    d, sc = x.cuda(), R.SCALES[scale]
    row, col = R.quantize_rows(x, scale), R.quantize_rows(x.t().contiguous(), scale)
    same(fp4.fp8_quantize(d, fp4.ROW, sc), *row, rows, cols)
    same(fp4.fp8_quantize(d, fp4.COL, sc), *col, cols, rows)
    r, c = fp4.fp8_quantize_rowcol(d, sc)
    same(r, *row, rows, cols)
    same(c, *col, cols, rows)
    q, qt, s = R.quantize_tiles(x, scale)
    f, t = fp4.fp8_quantize(d, fp4.TILE2D, sc)
    same(f, q, s, rows, cols)
    same(t, qt, s, cols, rows)
    assert (f.layout, t.layout) == (fp4.FP4_SCALES_2D, fp4.FP4_SCALES_2D_T)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_and_alignment(dtype):
    base = inputs(70, 400, dtype).cuda()
    for x in (base[:, 3:300], base[::2, :256], base[1:, 8:264]):
        r, c = fp4.fp8_quantize_rowcol(x)
        same(r, *R.quantize_rows(x.cpu(), "e8m0"), *x.shape)
        same(c, *R.quantize_rows(x.cpu().t().contiguous(), "e8m0"), x.shape[1], x.shape[0])


@pytest.mark.parametrize("scale", list(R.SCALES))
def test_extremes(scale):
    big, tiny = 3.0e38, 1.0e-45
    x = torch.zeros(8, 256)
    x[0, 0], x[0, 200] = big, -big
    x[1, 5] = tiny
    x[2, :128] = 1e-39
    x[3, 0] = 2.0 ** -100
    x[4, 0] = 2.0 ** -101
    x[5, 128:] = torch.linspace(-448, 448, 128)
    same(fp4.fp8_quantize(x.cuda(), fp4.ROW, R.SCALES[scale]), *R.quantize_rows(x, scale), 8, 256)


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_blocks_that_are_not_finite(scale, bad):
    x = R.randn(130, 300, 3)
    x[7, 130] = bad
    r, c = fp4.fp8_quantize_rowcol(x.cuda(), R.SCALES[scale])
    v, w = fp4.fp8_dequantize(r).cpu(), fp4.fp8_dequantize(c).cpu()
    block = torch.zeros(130, 300, dtype=torch.bool)
    block[7, 128:256] = True
    assert torch.equal(v.isnan(), block)
    block = torch.zeros(300, 130, dtype=torch.bool)
    block[130, :128] = True
    assert torch.equal(w.isnan(), block)
    one = R.scale_values(r.s)[7, 1], R.scale_values(c.s)[130, 0]
    assert one == (1.0, 1.0)
    ok = R.quantize_rows(torch.where(torch.isfinite(x), x, torch.zeros(())), scale)[0]
    assert torch.equal(r.q.cpu().view(torch.uint8)[8:], ok[8:])


def test_every_code_survives():
    codes = torch.arange(256, dtype=torch.uint8)
    codes = codes[(codes & 127) != 127]
    x = torch.zeros(1, 256)
    x[0, :codes.numel()] = codes.view(R.F8).float()
    x[0, 255] = 448.0   # both blocks hold 448, so both scales are one
    for scale in R.SCALES:
        t = fp4.fp8_quantize(x.cuda(), fp4.ROW, R.SCALES[scale])
        assert torch.equal(R.scale_values(t.s), torch.ones(1, 2, dtype=torch.float64))
        assert torch.equal(t.q.cpu().view(torch.uint8)[0, :codes.numel()], codes)


@pytest.mark.parametrize("layout", list(R.LAYOUTS))
@pytest.mark.parametrize("scale", list(R.SCALES))
def test_dequantize(layout, scale):
    t, v = R.operand(R.randn(150, 333, 5), layout, scale)
    assert torch.equal(fp4.fp8_dequantize(t).cpu(), v.float())   # a code times a float32 scale rounds once
    out = torch.zeros(150, 340, dtype=torch.bfloat16, device="cuda")
    fp4.fp8_dequantize(t, out=out[:, :333])
    assert torch.equal(out[:, :333].cpu(), v.float().to(torch.bfloat16)) and (out[:, 333:] == 0).all()


def test_mxfp4_to_fp8_is_an_operand():
    x = R.randn(48, 256, 9).cuda()
    y, s = fp4.mxfp4_to_fp8(fp4.quantize(x, fp4.E8M0, 32, fp4.ROW))
    t = fp4.F8Tensor(y, s, fp4.FP4_SCALES_1D, 48, 256)
    v = fp4.fp8_dequantize(t)
    assert torch.equal(v, fp4.dequantize(fp4.quantize(x, fp4.E8M0, 32, fp4.ROW)))   # exact within 14 binades
    w, wv = R.operand(R.randn(64, 256, 10), "2d", "e8m0")
    got = fp4.fp8_gemm(t, w, torch.float32).cpu().double()
    y64, tol = R.product_bound(v.cpu().double(), wv, torch.float32)
    assert ((got - y64).abs() <= tol).all()


def test_empty():
    for rows, cols in ((0, 256), (256, 0), (0, 0)):
        x = torch.zeros(rows, cols, device="cuda")
        for v in (fp4.ROW, fp4.COL):
            fp4.fp8_quantize(x, v)
        fp4.fp8_quantize(x, fp4.TILE2D)
        fp4.fp8_quantize_rowcol(x)


# ------------------------------------------------------------------ gated gradient

def grad64(dh, gu, kind):
    dh, f = dh.double(), dh.shape[1]
    g, u = gu[:, :f].double(), gu[:, f:].double()
    a, da = R.act(g, kind)
    return torch.cat([dh * u * da, dh * a], dim=1)


def grad_bound(d64, dh, gu, dtype):
    """Half a step of the output and the float32 arithmetic: exponential, reciprocal and error function within 4
    units and some six roundings, on terms of at most |dh| (1 + |u|) (1 + |g|) each."""
    f = dh.shape[1]
    g, u = gu[:, :f].double().abs(), gu[:, f:].double().abs()
    mag = torch.cat([dh.double().abs() * u * (1 + g), dh.double().abs() * (1 + g)], dim=1)
    return R.HALF[dtype] * d64.abs() + 2.0 ** -20 * mag + 2.0 ** -149


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,f", [(1, 1), (3, 7), (5, 128), (33, 1000), (130, 96)])
def test_gated_grad(rows, f, dtype, act):
    dh, gu = R.randn(rows, f, 1, dtype), R.randn(rows, 2 * f, 2, dtype, 4.0)
    d64 = grad64(dh, gu, act)
    got = fp4.gated_grad(dh.cuda(), gu.cuda(), act).cpu()
    assert got.dtype == dtype
    assert ((got.double() - d64).abs() <= grad_bound(d64, dh, gu, dtype)).all()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated_grad_matches_differences(act):
    """Against central differences of h = act(g) u in float64."""
    g = torch.linspace(-6, 6, 97, dtype=torch.float64)[None]
    u = torch.linspace(2, -2, 97, dtype=torch.float64)[None]
    e = 1e-5
    dg = (R.act(g + e, act)[0] - R.act(g - e, act)[0]) / (2 * e) * u
    du = (R.act(g, act)[0] * (u + e) - R.act(g, act)[0] * (u - e)) / (2 * e)
    got = fp4.gated_grad(torch.ones(1, 97, device="cuda"), torch.cat([g, u], 1).float().cuda(), act).cpu().double()
    # difference quotient: e^2 times the third derivative and 1e-16 / e; inputs rounded to 2^-24 of 6
    assert (got - torch.cat([dg, du], 1)).abs().max() < 4e-6


def test_gated_grad_far_inputs():
    """Gates far out on both sides: the slope is 0 or 1, nothing overflows into NaN."""
    g = torch.tensor([[-200.0, -100.0, -90.0, 90.0, 100.0, 200.0]])
    u, dh = torch.full_like(g, 2.0), torch.ones_like(g)
    want = torch.cat([torch.tensor([[0.0, 0, 0, 2, 2, 2]]), g.clamp_min(0)], 1)
    for act in ("silu", "gelu", "gelu_tanh"):
        got = fp4.gated_grad(dh.cuda(), torch.cat([g, u], 1).cuda(), act).cpu()
        assert torch.allclose(got, want, atol=1e-30)


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,f", [(1, 128), (77, 256), (300, 384)])
def test_fp8_gated_grad(rows, f, dtype, scale):
    dh, gu = R.randn(rows, f, 1, dtype, 1e-3).cuda(), R.randn(rows, 2 * f, 2, dtype, 2.0).cuda()
    # the same float32 gradient, so the same codes as quantizing a float32 call's result
    d = fp4.gated_grad(dh.float(), gu.float()).cpu()
    r, c = fp4.fp8_gated_grad(dh, gu, scale=R.SCALES[scale])
    same(r, *R.quantize_rows(d, scale), rows, 2 * f)
    same(c, *R.quantize_rows(d.t().contiguous(), scale), 2 * f, rows)
    r1, none = fp4.fp8_gated_grad(dh, gu, scale=R.SCALES[scale], col=False)
    assert none is None and torch.equal(r1.q.view(torch.uint8), r.q.view(torch.uint8))
    none, c1 = fp4.fp8_gated_grad(dh, gu, scale=R.SCALES[scale], row=False)
    assert none is None and torch.equal(c1.q.view(torch.uint8), c.q.view(torch.uint8))


def test_gated_grad_strides():
    dh, gu = R.randn(9, 300, 1).cuda(), R.randn(9, 700, 2).cuda()
    want = fp4.gated_grad(dh[:, 1:257].contiguous(), gu[:, 3:515].contiguous())
    out = torch.full((9, 600), 5.0, device="cuda")
    fp4.gated_grad(dh[:, 1:257], gu[:, 3:515], out=out[:, 5:517])
    assert torch.equal(out[:, 5:517], want) and (out[:, :5] == 5).all() and (out[:, 517:] == 5).all()
    r, c = fp4.fp8_gated_grad(dh[:, 1:257], gu[:, 3:515])
    r0, c0 = fp4.fp8_gated_grad(dh[:, 1:257].contiguous(), gu[:, 3:515].contiguous())
    assert torch.equal(r.q.view(torch.uint8), r0.q.view(torch.uint8)) and torch.equal(c.q.view(torch.uint8), c0.q.view(torch.uint8))
