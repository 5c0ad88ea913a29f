"""Every form of the 8-bit products (tests/_fp8_forms.py), exact on integers: sums below 2^24 of their unit, which both
matrix cores and any order of adding give exactly."""
import ctypes

import pytest
import torch

import fp4_block_scaled_tensor_amd as fp4
from fp4_block_scaled_tensor_amd import _lib
from tests import _fp8 as R
from tests import _fp8_forms as F
from tests.test_gpu_fp8_usage import Guarded

pytestmark = pytest.mark.gpu


def integers(rows, k, seed, layout, scale, least=-1):
    """An operand of integers -3 .. 3 with scales 2^least .. 2^(least + 2), and its float64 values, on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.zeros(rows, R.blocks(k) * R.B, device="cuda")
    q[:, :k] = torch.randint(-3, 4, (rows, k), generator=g, device="cuda").float()
    shape = (rows, R.blocks(k)) if layout == "1d" else (R.blocks(rows), R.blocks(k)) if layout == "2d" else (R.blocks(k), R.blocks(rows))
    e = torch.randint(least, least + 3, shape, generator=g, device="cuda")
    # (a table: the GPU's float64 power is off by a unit for some of these exponents)
    s = torch.tensor([2.0 ** (least + i) for i in range(3)], dtype=torch.float64, device="cuda")[e - least]
    held = (e + 127).to(torch.uint8) if scale == "e8m0" else s.float()
    if layout == "2dT":
        s = s.t()
    if layout != "1d":
        s = s.repeat_interleave(R.B, dim=0)[:rows]
    return fp4.F8Tensor(q.to(R.F8), held, R.LAYOUTS[layout], rows, k), q[:, :k].double() * s.repeat_interleave(R.B, dim=1)[:, :k]


def layouts(size):
    """All of them; of large weights one, and both kinds where the weight's scales may be turned too."""
    m, n, k, e = size
    if m * n * k < 2e10:
        return list(R.LAYOUTS)
    return ["1d", "2d"] if F.form(m, n, k, e, 0, 0)[3] else ["2d"]


def operands(size, layout, scale, least=-1):
    """x, the weight or stack, the first positions of the experts' rows (None: one weight), the product in float64."""
    m, n, k, e = size
    x, xv = integers(m, k, 1, layout="1d", scale=scale, least=least)
    if not e:
        w, wv = integers(n, k, 2, layout, scale)
        return x, w, None, xv @ wv.t().contiguous()
    share = torch.tensor([(1, 0, 3, 2, 7)[i % 5] for i in range(e)], dtype=torch.float64)
    ends = (share.cumsum(0) / share.sum() * (m - m // 16)).long()   # a sixteenth of the rows is dropped
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), ends])
    each, y = [], torch.zeros(m, n, dtype=torch.float64, device="cuda")
    for i in range(e):
        t, wv = integers(n, k, 10 + i, layout, scale)
        each.append(t)
        lo, hi = int(offsets[i]), int(offsets[i + 1])
        if hi > lo:
            y[lo:hi] = xv[lo:hi] @ wv.t().contiguous()
    return x, fp4.fp8_stack(each), offsets.to(torch.int32).cuda(), y


def name(size):
    return "x".join(map(str, size))


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("size", F.GEMM, ids=name)
def test_product(size, scale):
    for layout in layouts(size):
        x, w, offsets, y64 = operands(size, layout, scale)
        want = y64.float()
        assert torch.equal(want.double(), y64)
        for dtype in (torch.bfloat16, torch.float32):
            got = fp4.fp8_gemm(x, w, dtype) if offsets is None else fp4.fp8_expert_gemm(x, w, offsets, dtype)
            assert torch.equal(got, want.to(dtype)), (layout, dtype)


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("size", F.GATED, ids=name)
def test_gated(size, scale):
    """The projections exact, h against float64 within the activation's arithmetic, and h in bf16 and as codes what
    rounding or quantizing the float32 h gives."""
    for layout in layouts(size):
        x, w, offsets, gu64 = operands(size, layout, scale, least=-5)   # gates of a few units
        f = gu64.shape[1] // 2
        h, gu = fp4.fp8_gated(x, w, "silu", torch.float32, save=torch.float32, plan=offsets)
        assert torch.equal(gu.double(), gu64), layout
        g, u = gu64[:, :f], gu64[:, f:]
        h64 = g * torch.sigmoid(g) * u
        assert ((h.double() - h64).abs() <= 2.0 ** -20 * (1 + g.abs()) * u.abs() + 2.0 ** -24 * h64.abs()).all(), layout
        del h64, g, u
        want = fp4.fp8_quantize(h, fp4.ROW, R.SCALES[scale])
        for kept in (torch.bfloat16, torch.float32):
            q, gk = fp4.fp8_gated(x, w, "silu", torch.float8_e4m3fn, save=kept, plan=offsets)
            assert torch.equal(gk, gu.to(kept)), (layout, kept)
            assert torch.equal(q.q.view(torch.uint8), want.q.view(torch.uint8)), (layout, kept)
            assert torch.equal(q.s.view(torch.uint8), want.s.view(torch.uint8)), (layout, kept)
        assert torch.equal(fp4.fp8_gated(x, w, "silu", plan=offsets)[0], h.to(torch.bfloat16)), layout


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("size", [(3, 72, 300, 0), (9, 150, 640, 5), (70, 200, 1100, 0), (200, 528, 2048, 3), (700, 1040, 384, 0)], ids=name)
def test_gated_in_every_pair_of_types(size, scale):
    """h in each type, the projections in each or not kept, and each activation: all one result, rounded."""
    x, w, offsets, gu64 = operands(size, "2d", scale, least=-5)
    for act in ("silu", "gelu", "gelu_tanh"):
        h32, _ = fp4.fp8_gated(x, w, act, torch.float32, save=torch.float32, plan=offsets)
        codes = fp4.fp8_quantize(h32, fp4.ROW, R.SCALES[scale])
        for out in (torch.bfloat16, torch.float32, torch.float8_e4m3fn):
            for kept in (None, torch.bfloat16, torch.float32):
                h, gu = fp4.fp8_gated(x, w, act, out, save=kept, plan=offsets)
                assert gu is None if kept is None else torch.equal(gu, gu64.to(kept)), (act, out, kept)
                if out is torch.float8_e4m3fn:
                    assert torch.equal(h.q.view(torch.uint8), codes.q.view(torch.uint8)), (act, kept)
                    assert torch.equal(h.s.view(torch.uint8), codes.s.view(torch.uint8)), (act, kept)
                else:
                    assert torch.equal(h, h32.to(out)), (act, out, kept)


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("size,layout", [((17, 2050, 4096, 0), "2d"), ((2047, 200, 2048, 3), "2d"), ((4100, 70, 32768, 0), "1d"),
                                         ((4100, 70, 32768, 8), "2d"), ((4100, 4096, 14336, 0), "1d"), ((6144, 1030, 14336, 8), "1d")])
def test_workspaces_and_outputs_between_guards(size, layout, scale):
    """Split sums, turned scales and both in one workspace of exactly the bytes that are asked for; outputs exact."""
    m, n, k, e = size
    x, w, offsets, y64 = operands(size, layout, scale, least=-5)
    lib, nb, stream = _lib.load(), ctypes.c_size_t(), torch.cuda.current_stream().cuda_stream
    ox, ow = (_lib.F8Operand(t.q.data_ptr(), t.s.data_ptr(), R.SCALES[scale], t.layout, t.rows, t.k) for t in (x, w))
    off = None if offsets is None else offsets.data_ptr()
    for dt, dtype in ((0, torch.bfloat16), (1, torch.float32)):
        _lib.check(lib.fp8_gemm_workspace(m, ctypes.byref(ow), e, 0, dt, ctypes.byref(nb)))
        ws, y = Guarded(max(16, nb.value)), Guarded(m * n * dtype.itemsize)
        if e:
            _lib.check(lib.fp8_expert_gemm(ctypes.byref(ox), ctypes.byref(ow), e, off, y.ptr(), dt, n, ws.ptr(), nb.value, stream))
        else:
            _lib.check(lib.fp8_gemm(ctypes.byref(ox), ctypes.byref(ow), y.ptr(), dt, n, ws.ptr(), nb.value, stream))
        assert ws.intact() and y.intact()
        assert torch.equal(y.get(dtype).view(m, n), y64.float().to(dtype))
    kc = R.blocks(n // 2)
    _lib.check(lib.fp8_gemm_workspace(m, ctypes.byref(ow), e, 2, 0, ctypes.byref(nb)))
    ws, q, s = Guarded(max(16, nb.value)), Guarded(m * kc * R.B), Guarded(m * kc * (1 if scale == "e8m0" else 4))
    gu = Guarded(m * n * 2)
    _lib.check(lib.fp8_gated(ctypes.byref(ox), ctypes.byref(ow), e, off, 0, q.ptr(), _lib.FP8_OUT_E4M3, 0, s.ptr(), gu.ptr(), 0, n,
                             ws.ptr(), nb.value, stream))
    assert all(b.intact() for b in (ws, q, s, gu))
    assert torch.equal(gu.get(torch.bfloat16).view(m, n), y64.float().to(torch.bfloat16))
    codes = fp4.fp8_quantize(fp4.fp8_gated(x, w, "silu", torch.float32, plan=offsets)[0], fp4.ROW, R.SCALES[scale])
    assert torch.equal(q.get(), codes.q.view(torch.uint8).flatten()) and torch.equal(s.get(), codes.s.view(torch.uint8).flatten())
