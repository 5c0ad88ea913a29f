"""Forms of the mixture-of-experts operators that callers choose: outputs left out, no tensor scale or one per
stripe in a stack, no K, more choices to a token than partial sums are kept at a time, single 16-row bands."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import formats as OF
from test_gpu_experts import DT, HALF_ULP, U, close, gen, plain_sort, random_weight, router_ids, weight_from

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hidden", [72, 2052])
def test_combine_gradients_one_at_a_time(hidden, dtype):
    """dys without dw (ys NULL) and dw without dys (weights NULL) are those of the call for both, bit for bit."""
    from fp4_block_scaled_tensor_amd import _lib
    import fp4_block_scaled_tensor_amd as fp4
    tokens, topk, experts, dt = 19, 3, 5, DT[dtype]
    r = gen(hidden)
    ids = router_ids(r, tokens, topk, experts, 0.2)
    plan = fp4.expert_sort(torch.from_numpy(ids).cuda(), experts)
    dy = torch.from_numpy(r.standard_normal((tokens, hidden)).astype(np.float32)).to(dt).cuda()
    ys = torch.from_numpy(r.standard_normal((tokens * topk, hidden)).astype(np.float32)).to(dt).cuda()
    w = torch.from_numpy(r.standard_normal((tokens, topk)).astype(np.float32)).cuda()
    both = fp4.expert_combine_grad(dy, ys, w, plan)
    code = _lib.FP4_IN_FP32 if dt is torch.float32 else _lib.FP4_IN_BF16
    lib = fp4.library()

    def call(y, weights, dys, dw):
        p = lambda t: None if t is None else t.data_ptr()   # noqa: E731
        _lib.check(lib.fp4_expert_combine_grad(dy.data_ptr(), code, tokens, hidden, hidden, p(y), hidden, p(weights), topk,
                                               plan.pos.data_ptr(), topk, p(dys), hidden, p(dw), topk, None))
        torch.cuda.synchronize()
    dys = torch.full_like(both[0], float("nan"))
    call(None, w, dys, None)
    assert torch.equal(dys, both[0])
    dw = torch.full_like(both[1], float("nan"))
    call(ys, None, None, dw)
    assert torch.equal(dw, both[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("topk", [63, 64, 65, 130])
def test_many_choices_to_a_token(topk, dtype):
    """More choices than the weights' gradient keeps partial sums for at a time; experts may repeat in a token."""
    import fp4_block_scaled_tensor_amd as fp4
    tokens, experts, hidden, dt = 5, 9, 200, DT[dtype]
    r = gen(topk)
    ids = r.integers(-1, experts, (tokens, topk)).astype(np.int64)
    plan = fp4.expert_sort(torch.from_numpy(ids).cuda(), experts)
    order, pos, offsets = plain_sort(ids, experts)
    kept = offsets[-1]
    dy = torch.from_numpy(r.standard_normal((tokens, hidden)).astype(np.float32)).to(dt).cuda()
    ys = torch.from_numpy(r.standard_normal((tokens * topk, hidden)).astype(np.float32)).to(dt).cuda()
    w = r.standard_normal((tokens, topk)).astype(np.float32)
    wd = torch.from_numpy(w).cuda()
    dy64, y64 = dy.cpu().double().numpy(), ys.cpu().double().numpy()
    rows = np.where((pos >= 0)[:, :, None], y64[np.where(pos >= 0, pos, 0)], 0.0)

    terms = rows * w[:, :, None].astype(np.float64)
    got = fp4.expert_combine(ys, wd, plan).cpu().double().numpy()
    lim = (topk + 1) * 2 * U * np.abs(terms).sum(1) * 1.01 + HALF_ULP[dt] * np.abs(terms.sum(1)) * 1.01
    assert (np.abs(got - terms.sum(1)) <= lim).all(), "combine"
    dys, dw = fp4.expert_combine_grad(dy, ys, wd, plan)
    want = np.zeros((tokens * topk, hidden))
    want[:kept] = w.reshape(-1)[order[:kept]].astype(np.float64)[:, None] * dy64[order[:kept] // topk]
    assert (np.abs(dys.cpu().double().numpy() - want) <= (HALF_ULP[dt] + U) * np.abs(want) * 1.01).all(), "dys"
    prod = rows * dy64[:, None, :]
    assert (np.abs(dw.cpu().double().numpy() - prod.sum(2)) <= (hidden + 1) * U * np.abs(prod).sum(2) * 1.01).all(), "dw"


@pytest.mark.parametrize("m", [3, 40, 300])
def test_no_tensor_scale(m):
    """g NULL, or without elements in the binding, is 1: bit for bit the product with g = 1."""
    from fp4_block_scaled_tensor_amd import _lib
    import dataclasses
    import fp4_block_scaled_tensor_amd as fp4
    r, n, k = gen(m), 48, 320
    x = torch.from_numpy(r.standard_normal((m, k)).astype(np.float32)).to(torch.bfloat16).cuda()
    for fmt, block in (("ue5m3", 16), ("e8m0", 32)):
        w, _ = random_weight(r, n, k, fmt, block, "1d")
        want = fp4.linear(x, w)
        bare = dataclasses.replace(w, g=torch.empty(0, device="cuda"))
        assert torch.equal(fp4.linear(x, bare), want)
        y, nb = torch.empty_like(want), ctypes.c_size_t()
        op = _lib.Operand(w.q.data_ptr(), w.s.data_ptr(), None, w.fmt, w.block, w.layout, 0, n, k)
        _lib.check(fp4.library().fp4_linear_workspace(m, _lib.FP4_IN_BF16, ctypes.byref(op), 0, ctypes.byref(nb)))
        ws = torch.empty(max(16, nb.value), dtype=torch.uint8, device="cuda")
        _lib.check(fp4.library().fp4_linear(x.data_ptr(), _lib.FP4_IN_BF16, m, k, ctypes.byref(op), y.data_ptr(),
                                            _lib.FP4_IN_BF16, n, ws.data_ptr(), nb.value, None))
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("stripe", [16, 128])
@pytest.mark.parametrize("counts", [[2, 0, 1, 3], [30, 0, 70, 5], [1, 300, 0, 260]])
def test_stripes_in_a_stack(counts, stripe):
    """One tensor scale to a stripe of rows of each expert's weight."""
    import fp4_block_scaled_tensor_amd as fp4
    n, k, r = 200, 320, gen(stripe)
    pairs, gs = [], []
    for _ in counts:
        codes = r.integers(0, 16, (n, k)).astype(np.uint8)
        sc = (OF.SCALE_ONE_CODE[OF.E4M3] + r.integers(-8, 9, (n, k // 16))).astype(np.uint8)
        gs.append((r.random(-(-n // stripe)) + 0.5).astype(np.float32))
        pairs.append(weight_from(codes, sc, OF.E4M3, 16, "1d", gs[-1], g_stripe=stripe))
    ends = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x = torch.from_numpy(r.standard_normal((int(ends[-1]), k)).astype(np.float32)).to(torch.bfloat16).cuda()
    y = fp4.expert_linear(x, fp4.stack_experts([p[0] for p in pairs]), torch.from_numpy(ends).cuda(), out_dtype=torch.float32)
    for e, (_, w64) in enumerate(pairs):
        a, b = int(ends[e]), int(ends[e + 1])
        if a < b:
            close(y[a:b], x[a:b].cpu().double().numpy(), w64, np.repeat(gs[e], stripe)[:n].astype(np.float64)[None],
                  torch.float32, f"expert {e}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [0, 1, 70])
def test_no_k_gives_zeros(rows, dtype):
    import fp4_block_scaled_tensor_amd as fp4
    n = 48
    w = fp4.QTensor(torch.empty((n, 0), dtype=torch.uint8, device="cuda"), torch.empty((n, 0), dtype=torch.uint8,
                    device="cuda"), torch.full((1,), 3.0, device="cuda"), fp4.E8M0, 32, fp4.FP4_SCALES_1D, n, 0)
    x = torch.empty((rows, 0), dtype=DT[dtype], device="cuda")
    guard = torch.full((rows, n + 5), -7.0, dtype=DT[dtype], device="cuda")
    fp4.linear(x, w, out=guard[:, 2:2 + n])
    assert (guard[:, 2:2 + n] == 0).all() and (guard[:, :2] == -7).all() and (guard[:, 2 + n:] == -7).all()
    offsets = torch.tensor([0, rows // 2, rows - rows // 4], dtype=torch.int32, device="cuda")
    y = fp4.expert_linear(x, fp4.stack_experts([w, w]), offsets)
    assert y.shape == (rows, n) and (y == 0).all()


@pytest.mark.parametrize("m", [1, 5, 12, 40, 300])
@pytest.mark.parametrize("n", [16, 32])
@pytest.mark.parametrize("layout", ["2d", "2dT"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_band_of_a_two_dimensional_grid(dtype, layout, n, m):
    """2D scales of one or two bands of 16 weight rows, with a last half turn of K; exact on integers."""
    import fp4_block_scaled_tensor_amd as fp4
    r, k = gen(m + n), 448
    w, w64 = random_weight(r, n, k, "ue5m3", 16, layout, spread=1)
    x64 = r.integers(-8, 9, (m, k)).astype(np.float64)
    y = fp4.linear(torch.from_numpy(x64).to(DT[dtype]).cuda(), w, out_dtype=torch.float32)
    assert np.array_equal(y.cpu().double().numpy(), x64 @ w64.T)


@pytest.mark.parametrize("m", [4, 80])
@pytest.mark.parametrize("fmt,block", [("e8m0", 32), ("ue5m3", 16)])
def test_gradient_through_the_col_view(fmt, block, m):
    """A weight with 1D scales: dX = dY . W from the weight's COL view."""
    import fp4_block_scaled_tensor_amd as fp4
    r, n, k = gen(m), 192, 320
    w = torch.from_numpy(r.integers(-6, 7, (n, k)).astype(np.float32)).cuda()
    f = {"e8m0": fp4.E8M0, "ue5m3": fp4.UE5M3}[fmt]
    wt = fp4.quantize(w, f, block, fp4.COL, amax=None if fmt == "e8m0" else fp4.tensor_amax(w))
    w64 = fp4.dequantize(wt).double().cpu().numpy()              # [k, n]
    # the quantized weight is the weight to within half a step of E2M1 (2 between 4 and 6 sixths of the maximum) and
    # the rounding of a 3-mantissa-bit scale (a sixteenth)
    assert np.abs(w64 - w.cpu().double().numpy().T).max() <= 6 * (1 / 6 + 1 / 16)
    dy = r.integers(-4, 5, (m, n)).astype(np.float64)
    dx = fp4.linear(torch.from_numpy(dy).to(torch.bfloat16).cuda(), wt, out_dtype=torch.float32)
    close(dx, dy, w64, 1.0, torch.float32, "dx")
