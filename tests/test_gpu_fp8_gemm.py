"""fp8_gemm, fp8_expert_gemm and fp8_gated: exact on integers, against float64 otherwise."""
import pytest
import torch

import fp4_block_scaled_tensor_amd as fp4
from tests import _fp8 as R

pytestmark = pytest.mark.gpu

SIZES = [(1, 64, 128), (1, 33, 1), (3, 257, 130), (16, 512, 1024), (17, 300, 4096), (40, 256, 640), (64, 1000, 384),
         (100, 128, 2048), (129, 600, 129), (257, 513, 1000), (300, 2048, 512), (700, 700, 700)]


def close(got, want, tol):
    got = got.cpu().double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} off, worst {((got - want).abs() - tol).max():.3g}"


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("layout", list(R.LAYOUTS))
@pytest.mark.parametrize("m,n,k", SIZES)
def test_gemm_exact_on_integers(m, n, k, layout, scale):
    a, av = R.integers(m, k, 1, "1d", scale)
    b, bv = R.integers(n, k, 2, layout, scale)
    want = (av @ bv.t()).float()
    assert torch.equal(fp4.fp8_gemm(a, b, torch.float32).cpu(), want)
    assert torch.equal(fp4.fp8_gemm(a, b).cpu(), want.to(torch.bfloat16))


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("layout", list(R.LAYOUTS))
@pytest.mark.parametrize("m,n,k", [(1, 200, 4096), (20, 513, 1000), (200, 300, 3000), (600, 520, 2047)])
def test_gemm_against_float64(m, n, k, layout, scale):
    a, av = R.operand(R.randn(m, k, 3) * torch.pow(2.0, 4 * R.randn(m, 1, 4)), "1d", scale)
    b, bv = R.operand(0.02 * R.randn(n, k, 5), layout, scale)
    for dtype in (torch.float32, torch.bfloat16):
        close(fp4.fp8_gemm(a, b, dtype), *R.product_bound(av, bv, dtype))
    y = fp4.fp8_gemm(a, b, torch.float32).cpu().double()
    assert (y - av @ bv.t()).norm() <= 1e-6 * (av @ bv.t()).norm()


@pytest.mark.parametrize("scale", list(R.SCALES))
def test_training_step_of_a_linear_layer(scale):
    """Quantize, forward, both gradients, as a layer runs them."""
    tokens, hidden, out = 333, 500, 640
    sc = R.SCALES[scale]
    x, dy = R.randn(tokens, hidden, 1, torch.bfloat16).cuda(), R.randn(tokens, out, 2, torch.bfloat16, 1e-3).cuda()
    w = R.randn(out, hidden, 3, std=0.02).cuda()
    xr, xc = fp4.fp8_quantize_rowcol(x, sc)
    dr, dc = fp4.fp8_quantize_rowcol(dy, sc)
    wf, wt = fp4.fp8_quantize(w, fp4.TILE2D, sc)
    v = lambda t: fp4.fp8_dequantize(t).cpu().double()   # noqa: E731
    for a, b, dtype in ((xr, wf, torch.bfloat16), (dr, wt, torch.bfloat16), (dc, xc, torch.float32)):
        close(fp4.fp8_gemm(a, b, dtype), *R.product_bound(v(a), v(b), dtype))


def test_gemm_into_strided_rows():
    a, av = R.integers(37, 256, 1, "1d", "e8m0")
    b, bv = R.integers(301, 256, 2, "2d", "e8m0")
    want = (av @ bv.t()).float()
    for dtype in (torch.float32, torch.bfloat16):
        for lead, ld in ((0, 304), (1, 310), (8, 320)):
            out = torch.full((39, ld), 9.0, dtype=dtype, device="cuda")
            fp4.fp8_gemm(a, b, out=out[1:38, lead:lead + 301])
            assert torch.equal(out[1:38, lead:lead + 301].cpu(), want.to(dtype))
            out[1:38, lead:lead + 301] = 9.0
            assert (out == 9.0).all()


def test_gemm_empty_and_no_k():
    for m, n, k in ((0, 64, 128), (5, 0, 128), (5, 70, 0), (300, 300, 0)):
        a, _ = R.integers(m, k, 1, "1d", "e8m0")
        b, _ = R.integers(n, k, 2, "2d", "e8m0")
        y = fp4.fp8_gemm(a, b)
        assert y.shape == (m, n) and (y == 0).all()


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("m", [3, 200])
def test_nan_stays_in_its_row(scale, m):
    x = R.randn(m, 400, 1)
    x[2, 399] = float("nan")
    a = fp4.fp8_quantize(x.cuda(), fp4.ROW, R.SCALES[scale])
    b, _ = R.operand(R.randn(300, 400, 2), "2d", scale)
    y = fp4.fp8_gemm(a, b)
    assert y[2].isnan().all() and not y[:2].isnan().any() and not y[3:].isnan().any()


@pytest.mark.parametrize("m", [1, 20, 150])
def test_far_scales(m):
    """E8M0 codes at both ends, float32 scales far apart: products within float32."""
    a, _ = R.integers(m, 384, 1, "1d", "e8m0")
    b, _ = R.integers(70, 384, 2, "1d", "e8m0")
    a.s[:] = torch.tensor([0, 127, 254], dtype=torch.uint8, device="cuda")
    b.s[:] = torch.tensor([254, 127, 0], dtype=torch.uint8, device="cuda")
    av = R.values(a.q, a.s, "1d", m, 384)
    bv = R.values(b.q, b.s, "1d", 70, 384)
    close(fp4.fp8_gemm(a, b, torch.float32), *R.product_bound(av, bv, torch.float32))
    f = lambda t: fp4.F8Tensor(t.q, R.scale_values(t.s).float().cuda(), t.layout, t.rows, t.k)   # noqa: E731
    close(fp4.fp8_gemm(f(a), f(b), torch.float32), *R.product_bound(av, bv, torch.float32))


def test_equal_calls_give_equal_bits():
    for m, n, k in ((1, 4096, 4096), (50, 640, 8192), (500, 700, 4096)):
        a, _ = R.operand(R.randn(m, k, 1), "1d", "f32")
        b, _ = R.operand(R.randn(n, k, 2), "2d", "f32")
        y = fp4.fp8_gemm(a, b, torch.float32)
        for _ in range(3):
            assert torch.equal(fp4.fp8_gemm(a, b, torch.float32), y)


# ------------------------------------------------------------------ experts

def stack(n_experts, n, k, layout, scale):
    each = [R.integers(n, k, 100 + e, layout, scale) for e in range(n_experts)]
    return fp4.fp8_stack([t for t, _ in each]), [v for _, v in each]


def experts64(xv, wv, offsets):
    y = torch.zeros(xv.shape[0], wv[0].shape[0], dtype=torch.float64)
    for e in range(len(wv)):
        y[offsets[e]:offsets[e + 1]] = xv[offsets[e]:offsets[e + 1]] @ wv[e].t()
    return y


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("layout", ["1d", "2d", "2dT"])
@pytest.mark.parametrize("counts,rows,n,k", [
    ([1], 1, 100, 256), ([0, 3, 0, 2], 7, 130, 300), ([5, 0, 40, 1, 0, 17, 9, 30], 110, 300, 640),
    ([300, 0, 129, 71], 512, 257, 384), ([0, 0, 0], 20, 64, 128), ([2] * 70, 150, 96, 128)])
def test_experts_exact_on_integers(counts, rows, n, k, layout, scale):
    x, xv = R.integers(rows, k, 1, "1d", scale)
    w, wv = stack(len(counts), n, k, layout, scale)
    offsets = torch.tensor([0] + counts).cumsum(0)
    want = experts64(xv, wv, offsets.tolist()).float()
    off = offsets.to(torch.int32).cuda()
    assert torch.equal(fp4.fp8_expert_gemm(x, w, off, torch.float32).cpu(), want)
    assert torch.equal(fp4.fp8_expert_gemm(x, w, off).cpu(), want.to(torch.bfloat16))


def test_experts_as_a_layer_runs_them():
    """sort -> gather of codes and scales -> product -> combine."""
    tokens, topk, n_experts, hidden, n = 150, 2, 5, 512, 320
    g = torch.Generator().manual_seed(0)
    ids = torch.randint(0, n_experts, (tokens, topk), generator=g)
    ids[7, 1] = -1
    plan = fp4.expert_sort(ids.cuda(), n_experts)
    x = R.randn(tokens, hidden, 1, torch.bfloat16)
    xs = fp4.fp8_quantize(fp4.expert_gather(x.cuda(), plan), fp4.ROW)
    w, wv = stack(n_experts, n, hidden, "2d", "e8m0")
    ys = fp4.fp8_expert_gemm(xs, w, plan)
    weights = torch.rand(tokens, topk, generator=g).cuda()
    y = fp4.expert_combine(ys, weights, plan).cpu().double()
    q, s = R.quantize_rows(x, "e8m0")
    xv = R.values(q, s, "1d", tokens, hidden)
    for t in range(tokens):
        want, mag = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
        for j in range(topk):
            if ids[t, j] >= 0:
                v, c = wv[ids[t, j]], weights[t, j].double().cpu()
                want += c * (xv[t] @ v.t())
                mag += c * (xv[t].abs() @ v.abs().t())
        assert ((y[t] - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -13) * mag).all()


# ------------------------------------------------------------------ gated

def gated64(xv, wv, kind):
    gu = xv @ wv.t()
    f = wv.shape[0] // 2
    return R.act(gu[:, :f], kind)[0] * gu[:, f:], gu


def gated_bound(xv, wv, h64, gu64, dtype):
    """The projections' bounds through the activation (slope at most 1.2) and the product, and float32 roundings.
    dtype: float32 where they are sums of the bf16 core (h or gu float32), else those of the E4M3 core."""
    f = wv.shape[0] // 2
    d = R.product_bound(xv, wv, dtype)[1] - (R.HALF[dtype] - R.HALF[torch.float32]) * gu64.abs()
    g, u = gu64[:, :f].abs(), gu64[:, f:].abs()
    return 1.2 * d[:, :f] * (u + d[:, f:]) + g * d[:, f:] + 2.0 ** -20 * (1 + g) * u


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("layout", list(R.LAYOUTS))
@pytest.mark.parametrize("m,f,k", [(1, 64, 128), (4, 1000, 4096), (17, 130, 300), (33, 40, 1000), (130, 128, 640), (300, 300, 700),
                                   (260, 1024, 384)])
def test_gated(m, f, k, layout, scale):
    x, xv = R.operand(R.randn(m, k, 1), "1d", scale)
    w, wv = R.operand(R.randn(2 * f, k, 2, std=2 / k ** 0.5), layout, scale)
    for act in ("silu", "gelu", "gelu_tanh"):
        h64, gu64 = gated64(xv, wv, act)
        fine, coarse = (gated_bound(xv, wv, h64, gu64, t) for t in (torch.float32, torch.bfloat16))
        h, none = fp4.fp8_gated(x, w, act, torch.float32)
        assert none is None
        close(h, h64, fine + R.HALF[torch.float32] * h64.abs())
        h, gu = fp4.fp8_gated(x, w, act, torch.bfloat16, save=torch.float32)
        close(h, h64, fine + R.HALF[torch.bfloat16] * h64.abs())
        close(gu, *R.product_bound(xv, wv, torch.float32))
        h, gu = fp4.fp8_gated(x, w, act, torch.bfloat16, save=torch.bfloat16)
        close(h, h64, coarse + R.HALF[torch.bfloat16] * h64.abs())
        close(gu, *R.product_bound(xv, wv, torch.bfloat16))
        h, gu = fp4.fp8_gated(x, w, act, torch.float8_e4m3fn, save=torch.bfloat16)
        close(gu, *R.product_bound(xv, wv, torch.bfloat16))
        assert (h.rows, h.k, h.layout) == (m, f, fp4.FP4_SCALES_1D)
        R.close_codes(fp4.fp8_dequantize(h), h64, coarse)


def codes_of(h, q, scale):
    """q holds exactly the codes and scales of the float32 h."""
    cq, cs = R.quantize_rows(h.cpu(), scale)
    assert torch.equal(q.q.cpu().view(torch.uint8), cq)
    assert torch.equal(q.s.cpu() if scale == "f32" else q.s.cpu().view(torch.uint8), cs)


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("m,f,k", [(1, 130, 256), (5, 77, 4096), (20, 300, 640), (70, 128, 1000), (150, 513, 128), (520, 640, 130)])
def test_gated_codes_exact_on_integers(m, f, k, scale):
    """Sums that are exact on both matrix cores: the codes are those of the float32 h, the projections are equal."""
    x, xv = R.integers(m, k, 1, "1d", scale)
    w, wv = R.integers(2 * f, k, 2, "2d", scale)
    x.s, xv = (x.s.view(torch.uint8) - 4 if scale == "e8m0" else x.s / 16), xv / 16   # gates of a few units
    for act in ("silu", "gelu", "gelu_tanh"):
        h, gu = fp4.fp8_gated(x, w, act, torch.float32, save=torch.float32)
        assert torch.equal(gu.cpu(), (xv @ wv.t()).float())
        q, gb = fp4.fp8_gated(x, w, act, torch.float8_e4m3fn, save=torch.bfloat16)
        assert torch.equal(gb, gu.to(torch.bfloat16))
        codes_of(h, q, scale)
        assert torch.equal(fp4.fp8_gated(x, w, act)[0], h.to(torch.bfloat16))


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("counts,rows,f,k", [([0, 3, 0, 2], 7, 70, 300), ([150, 0, 40, 1, 60], 300, 200, 256)])
def test_gated_experts(counts, rows, f, k, scale):
    x, xv = R.operand(R.randn(rows, k, 1), "1d", scale)
    each = [R.operand(R.randn(2 * f, k, 50 + e, std=2 / k ** 0.5), "2d", scale) for e in range(len(counts))]
    w = fp4.fp8_stack([t for t, _ in each])
    off = torch.tensor([0] + counts).cumsum(0)
    h, gu = fp4.fp8_gated(x, w, "silu", torch.float32, save=torch.float32, plan=off.to(torch.int32).cuda())
    q, gb = fp4.fp8_gated(x, w, "silu", torch.float8_e4m3fn, save=torch.bfloat16, plan=off.to(torch.int32).cuda())
    qv = fp4.fp8_dequantize(q)
    for e in range(len(counts)):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            h64, gu64 = gated64(xv[lo:hi], each[e][1], "silu")
            fine, coarse = (gated_bound(xv[lo:hi], each[e][1], h64, gu64, t) for t in (torch.float32, torch.bfloat16))
            close(h[lo:hi], h64, fine + R.HALF[torch.float32] * h64.abs())
            close(gu[lo:hi], *R.product_bound(xv[lo:hi], each[e][1], torch.float32))
            close(gb[lo:hi], *R.product_bound(xv[lo:hi], each[e][1], torch.bfloat16))
            R.close_codes(qv[lo:hi], h64, coarse)
    for t in (h, gu, gb, qv):
        assert (t[off[-1]:] == 0).all()
    assert (R.scale_values(q.s)[off[-1]:] == 1).all()


def test_gated_no_k():
    x, _ = R.integers(5, 0, 1, "1d", "e8m0")
    w, _ = R.integers(300, 0, 2, "2d", "e8m0")
    h, gu = fp4.fp8_gated(x, w, save=torch.float32)
    assert (h == 0).all() and (gu == 0).all()
    q, _ = fp4.fp8_gated(x, w, "silu", torch.float8_e4m3fn)
    assert (q.q.view(torch.uint8) == 0).all() and (q.s.view(torch.uint8) == 127).all()


@pytest.mark.parametrize("scale", list(R.SCALES))
def test_gated_block_forward_and_backward(scale):
    """A gated feed-forward block's training step: every product and gradient against float64 on the operands that the
    step itself quantized."""
    tokens, hidden, f = 260, 384, 256
    sc = R.SCALES[scale]
    x = R.randn(tokens, hidden, 1, torch.bfloat16).cuda()
    w1, w2 = R.randn(2 * f, hidden, 2, std=0.05).cuda(), R.randn(hidden, f, 3, std=0.05).cuda()
    dy = R.randn(tokens, hidden, 4, torch.bfloat16, 1e-3).cuda()
    v = lambda t: fp4.fp8_dequantize(t).cpu().double()   # noqa: E731
    xr, xc = fp4.fp8_quantize_rowcol(x, sc)
    w1f, w1t = fp4.fp8_quantize(w1, fp4.TILE2D, sc)
    w2f, w2t = fp4.fp8_quantize(w2, fp4.TILE2D, sc)
    h, gu = fp4.fp8_gated(xr, w1f, "silu", torch.float8_e4m3fn, save=torch.bfloat16)
    close(fp4.fp8_gemm(h, w2f), *R.product_bound(v(h), v(w2f), torch.bfloat16))
    dyr = fp4.fp8_quantize(dy, fp4.ROW, sc)
    dh = fp4.fp8_gemm(dyr, w2t)
    close(dh, *R.product_bound(v(dyr), v(w2t), torch.bfloat16))
    dr, dc = fp4.fp8_gated_grad(dh, gu, "silu", sc)
    g, u = gu[:, :f].cpu().double(), gu[:, f:].cpu().double()
    a, da = R.act(g, "silu")
    want = torch.cat([dh.cpu().double() * u * da, dh.cpu().double() * a], 1)
    R.close_codes(v(dr), want, 2.0 ** -16 * want.abs())
    R.close_codes(v(dc), want.t().contiguous(), 2.0 ** -16 * want.t().abs())
    close(fp4.fp8_gemm(dr, w1t), *R.product_bound(v(dr), v(w1t), torch.bfloat16))
    close(fp4.fp8_gemm(dc, xc, torch.float32), *R.product_bound(v(dc), v(xc), torch.float32))
