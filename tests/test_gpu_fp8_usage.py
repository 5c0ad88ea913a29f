"""The 8-bit operators as a program uses them: every tile form, captured and replayed, on other streams and
threads, into guarded buffers, at sizes past 32-bit offsets."""
import threading

import pytest
import torch

import fp4_block_scaled_tensor_amd as fp4
from fp4_block_scaled_tensor_amd import _lib
from tests import _fp8 as R

pytestmark = pytest.mark.gpu


def gpu_values(t):
    """An operand's float64 values, on the GPU."""
    v = t.q.view(torch.uint8).view(R.F8).double()[:, :t.k]
    s = R.scale_values(t.s).cuda()
    if t.layout == fp4.FP4_SCALES_2D_T:
        s = s.t()
    if t.layout != fp4.FP4_SCALES_1D:
        s = s.repeat_interleave(R.B, dim=0)[:t.rows]
    return v * s.repeat_interleave(R.B, dim=1)[:, :t.k]


def integers(rows, k, seed, layout, scale):
    """As R.integers, drawn on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.zeros(rows, R.blocks(k) * R.B, device="cuda")
    q[:, :k] = torch.randint(-3, 4, (rows, k), generator=g, device="cuda").float()
    shape = (rows, R.blocks(k)) if layout == "1d" else (R.blocks(rows), R.blocks(k)) if layout == "2d" else (R.blocks(k), R.blocks(rows))
    e = torch.randint(-1, 2, shape, generator=g, device="cuda")
    s = (e + 127).to(torch.uint8) if scale == "e8m0" else torch.pow(2.0, e.double()).float()
    return fp4.F8Tensor(q.to(R.F8), s, R.LAYOUTS[layout], rows, k)


# sums of integers times 2^-2 .. 2^2, below 2^22 in quarters: exact in float32
FORMS = [(2100, 4200, 640), (1000, 6144, 2048), (515, 1030, 1100), (200, 2100, 1100), (90, 700, 3000), (2048, 28672, 6144)]


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("layout", list(R.LAYOUTS))
@pytest.mark.parametrize("m,n,k", FORMS)
def test_gemm_forms_exact_on_integers(m, n, k, layout, scale):
    a, b = integers(m, k, 1, "1d", scale), integers(n, k, 2, layout, scale)
    want = gpu_values(a) @ gpu_values(b).t().contiguous()
    assert torch.equal(fp4.fp8_gemm(a, b, torch.float32), want.float())
    assert torch.equal(fp4.fp8_gemm(a, b), want.float().to(torch.bfloat16))


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("layout", ["1d", "2d"])
@pytest.mark.parametrize("m,f,k", [(2100, 2100, 640), (1000, 4096, 2048), (515, 518, 1100), (200, 1050, 1100), (90, 350, 3000)])
def test_gated_forms_exact_on_integers(m, f, k, layout, scale):
    x, w = integers(m, k, 1, "1d", scale), integers(2 * f, k, 2, layout, scale)
    x.s = x.s.view(torch.uint8) - 4 if scale == "e8m0" else x.s / 16   # gates of a few units
    gu64 = gpu_values(x) @ gpu_values(w).t().contiguous()
    h, gu = fp4.fp8_gated(x, w, "silu", torch.float32, save=torch.float32)
    assert torch.equal(gu, gu64.float())
    g, u = gu64[:, :f], gu64[:, f:]
    h64 = g * torch.sigmoid(g) * u
    assert ((h.double() - h64).abs() <= 2.0 ** -20 * (1 + g.abs()) * u.abs() + 2.0 ** -24 * h64.abs()).all()
    q, gb = fp4.fp8_gated(x, w, "silu", torch.float8_e4m3fn, save=torch.bfloat16)
    assert torch.equal(gb, gu.to(torch.bfloat16))
    cq, cs = R.quantize_rows(h.cpu(), scale)
    assert torch.equal(q.q.cpu().view(torch.uint8), cq)
    assert torch.equal(q.s.cpu() if scale == "f32" else q.s.cpu().view(torch.uint8), cs)
    assert torch.equal(fp4.fp8_gated(x, w)[0], h.to(torch.bfloat16))


@pytest.mark.parametrize("scale", list(R.SCALES))
@pytest.mark.parametrize("counts,rows,n,k", [([900, 0, 1400, 33], 2400, 2100, 640), ([300, 5, 0, 800], 1200, 4096, 1024),
                                             ([1] * 100 + [60], 170, 200, 384)])
def test_expert_forms_exact_on_integers(counts, rows, n, k, scale):
    x = integers(rows, k, 1, "1d", scale)
    each = [integers(n, k, 10 + e, "2d", scale) for e in range(len(counts))]
    w, off = fp4.fp8_stack(each), torch.tensor([0] + counts).cumsum(0)
    want = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    for e, t in enumerate(each):
        want[off[e]:off[e + 1]] = gpu_values(x)[off[e]:off[e + 1]] @ gpu_values(t).t().contiguous()
    off = off.to(torch.int32).cuda()
    assert torch.equal(fp4.fp8_expert_gemm(x, w, off, torch.float32), want.float())
    assert torch.equal(fp4.fp8_expert_gemm(x, w, off), want.float().to(torch.bfloat16))


# ------------------------------------------------------------------ graphs, streams, threads

def step(s):
    """A gated block's training step over static inputs; what it gives, by name."""
    xr, xc = fp4.fp8_quantize_rowcol(s["x"])
    h, gu = fp4.fp8_gated(xr, s["w1"], "silu", torch.float8_e4m3fn, save=torch.bfloat16)
    y = fp4.fp8_gemm(h, s["w2"])
    dyr, dyc = fp4.fp8_quantize_rowcol(s["dy"])
    dr, dc = fp4.fp8_gated_grad(fp4.fp8_gemm(dyr, s["w2t"]), gu)
    ys = fp4.fp8_expert_gemm(xr, s["we"], s["offsets"])
    one, _ = fp4.fp8_gated(fp4.fp8_quantize(s["x"][:3]), s["w1"], "gelu")
    return dict(y=y, dx=fp4.fp8_gemm(dr, s["w1t"]), dw=fp4.fp8_gemm(dc, xc, torch.float32), ys=ys, one=one,
                h=h.q.view(torch.uint8), hs=h.s.view(torch.uint8), gu=gu, back=fp4.fp8_dequantize(dyc))


def state(seed, tokens=300, hidden=1024, f=512):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *n: torch.randn(*n, generator=g).cuda()   # noqa: E731
    w1, w1t = fp4.fp8_quantize(0.05 * rand(2 * f, hidden), fp4.TILE2D)
    w2, w2t = fp4.fp8_quantize(0.05 * rand(hidden, f), fp4.TILE2D)
    we = fp4.fp8_stack([fp4.fp8_quantize(0.05 * rand(640, hidden), fp4.TILE2D)[0] for _ in range(3)])
    return dict(x=rand(tokens, hidden).bfloat16(), dy=(1e-3 * rand(tokens, hidden)).bfloat16(), w1=w1, w1t=w1t, w2=w2,
                w2t=w2t, we=we, offsets=torch.tensor([0, 90, 90, 280], dtype=torch.int32, device="cuda"))


def same(a, b):
    return all(torch.equal(a[k], b[k]) for k in a)


def test_captured_and_replayed():
    s = state(0)
    inputs = [{k: state(i)[k] for k in ("x", "dy")} for i in range(3)]
    want = []
    for i in inputs:
        for k in i:
            s[k].copy_(i[k])
        want.append({k: v.clone() for k, v in step(s).items()})
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(s)
    for n in (0, 1, 2, 1, 0):
        for k in inputs[n]:
            s[k].copy_(inputs[n][k])
        graph.replay()
        eager = fp4.fp8_gemm(fp4.fp8_quantize(s["x"]), s["w1"])   # the program's own work between replays
        torch.cuda.synchronize()
        assert same(out, want[n])
        assert eager.shape == (300, 1024)


def test_two_graphs_at_once():
    """Two captures of the same step (each has its own workspaces), replayed on two streams together."""
    states, graphs, outs, want = [state(i) for i in range(2)], [], [], []
    for s in states:
        want.append({k: v.clone() for k, v in step(s).items()})
    torch.cuda.synchronize()
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(s))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert same(outs[0], want[0]) and same(outs[1], want[1])


def test_threads_on_their_own_streams():
    states = [state(i) for i in range(4)]
    want = [{k: v.clone() for k, v in step(s).items()} for s in states]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(8):
                    got = step(states[i])
                    stream.synchronize()
                    if not same(got, want[i]):
                        bad.append(i)
        except Exception as e:   # noqa: BLE001
            bad.append(repr(e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


# ------------------------------------------------------------------ guarded buffers

class Guarded:
    """A buffer of n bytes between 4 KiB of a pattern."""

    def __init__(self, n):
        self.n, self.all = n, torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")

    def ptr(self):
        return self.all.data_ptr() + 4096

    def get(self, dtype=torch.uint8):
        return self.all[4096:4096 + self.n].clone().view(dtype)

    def intact(self):
        return bool((self.all[:4096] == 0xA5).all() and (self.all[4096 + self.n:] == 0xA5).all())


@pytest.mark.parametrize("scale", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols,lead", [(1, 1, 0), (3, 130, 0), (129, 257, 1), (128, 128, 0), (300, 7, 3), (5, 1000, 0)])
def test_quantize_writes_its_outputs_only(rows, cols, lead, dtype, scale):
    lib, es, code = _lib.load(), 1 if scale == 0 else 4, 1 if dtype == torch.float32 else 0
    x = R.randn(rows, cols + lead, 1, dtype).cuda()[:, lead:]
    kr, kc = R.blocks(cols), R.blocks(rows)
    for view in (0, 1, 2, 3):
        q, qt = Guarded(rows * kr * 128), Guarded(cols * kc * 128)
        s = Guarded((kc if view == 2 else rows) * kr * es)
        st = Guarded(cols * kc * es)
        _lib.check(lib.fp8_quantize(x.data_ptr(), code, rows, cols, x.stride(0), view, scale, q.ptr(), s.ptr(), qt.ptr(), st.ptr(),
                                    torch.cuda.current_stream().cuda_stream))
        assert all(g.intact() for g in (q, qt, s, st))
        t = fp4.fp8_quantize(x.contiguous(), (0, 1, 2, 0)[view], scale)
        if view in (0, 3):
            assert torch.equal(q.get(), t.q.view(torch.uint8).flatten())
        if view == 1:
            assert torch.equal(qt.get(), t.q.view(torch.uint8).flatten())
        if view == 2:
            assert torch.equal(q.get(), t[0].q.view(torch.uint8).flatten()) and torch.equal(qt.get(), t[1].q.view(torch.uint8).flatten())


@pytest.mark.parametrize("scale", ["e8m0", "f32"])
@pytest.mark.parametrize("m,f,k", [(1, 40, 256), (5, 130, 300), (70, 200, 640), (260, 1000, 384)])
def test_products_write_their_outputs_only(m, f, k, scale):
    """h's codes and scales, the projections and a plain product, between guards; workspaces of exactly what is asked."""
    import ctypes
    lib = _lib.load()
    x, _ = R.operand(R.randn(m, k, 1), "1d", scale)
    w, _ = R.operand(R.randn(2 * f, k, 2), "2d", scale)
    sc, es = R.SCALES[scale], 1 if scale == "e8m0" else 4
    ox = _lib.F8Operand(x.q.data_ptr(), x.s.data_ptr(), sc, x.layout, m, k)
    ow = _lib.F8Operand(w.q.data_ptr(), w.s.data_ptr(), sc, w.layout, 2 * f, k)
    nb = ctypes.c_size_t()
    stream = torch.cuda.current_stream().cuda_stream
    _lib.check(lib.fp8_gemm_workspace(m, ctypes.byref(ow), 0, 2, 0, ctypes.byref(nb)))
    ws, q, s, gu = Guarded(max(16, nb.value)), Guarded(m * R.blocks(f) * 128), Guarded(m * R.blocks(f) * es), Guarded(m * 2 * f * 2)
    _lib.check(lib.fp8_gated(ctypes.byref(ox), ctypes.byref(ow), 0, None, 0, q.ptr(), 2, 0, s.ptr(), gu.ptr(), 0, 2 * f, ws.ptr(),
                             nb.value, stream))
    assert all(g.intact() for g in (ws, q, s, gu))
    h, g = fp4.fp8_gated(x, w, "silu", torch.float8_e4m3fn, save=torch.bfloat16)
    assert torch.equal(q.get(), h.q.view(torch.uint8).flatten()) and torch.equal(gu.get(torch.bfloat16), g.flatten())
    for dt, size in ((0, 2), (1, 4)):
        _lib.check(lib.fp8_gemm_workspace(m, ctypes.byref(ow), 0, 0, dt, ctypes.byref(nb)))
        ws, y = Guarded(max(16, nb.value)), Guarded(m * 2 * f * size)
        _lib.check(lib.fp8_gemm(ctypes.byref(ox), ctypes.byref(ow), y.ptr(), dt, 2 * f, ws.ptr(), nb.value, stream))
        assert ws.intact() and y.intact()


# ------------------------------------------------------------------ large

def test_operands_past_four_gigabytes():
    """A weight of 4.6e9 bytes and an output whose last rows lie past 2^32 bytes, by few rows and by tiles."""
    n, k = (1 << 20) + 77, 4352
    w = fp4.F8Tensor(torch.zeros(n, k, dtype=torch.uint8, device="cuda"), torch.full((R.blocks(n), k // 128), 127, dtype=torch.uint8, device="cuda"),
                     fp4.FP4_SCALES_2D, n, k)
    for r, c in ((0, 0), (n - 1, k - 1), (n - 1, 0), (n // 2, 5)):
        w.q[r, c] = 0x38   # one
    for m in (2, 1030):
        x = integers(m, k, 3, "1d", "e8m0")
        xv = gpu_values(x)
        y = fp4.fp8_gemm(x, w)
        want = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
        for r, cols in ((0, [0]), (n // 2, [5]), (n - 1, [0, k - 1])):
            want[:, r] = xv[:, cols].sum(dim=1).to(torch.bfloat16)
        assert torch.equal(y, want)
        del y, want


def test_quantize_past_four_gigabytes():
    rows, cols = 40003, 30000
    x = torch.zeros(rows, cols, device="cuda")
    x[0, 0], x[rows - 1, cols - 1], x[rows - 1, 0], x[rows // 2, 777] = 1.0, -3.0, 448.0, 2.0
    r, c = fp4.fp8_quantize_rowcol(x)
    for t, v in ((r, x), (c, x.t())):
        for i, j in ((0, 0), (t.rows - 1, t.k - 1), (t.rows - 1, 0), (0, t.k - 1), (rows // 2, 777), (777, rows // 2)):
            if i < t.rows and j < t.k:
                code = t.q[i:i + 1, j // 128 * 128:j // 128 * 128 + 128]
                want, s = R.quantize_rows(v[i:i + 1, j // 128 * 128:j // 128 * 128 + 128].cpu(), "e8m0")
                assert torch.equal(code.cpu().view(torch.uint8), want)
                assert t.s.view(torch.uint8)[i, j // 128].item() == s[0, 0].item()
        assert int((t.q.view(torch.uint8) != 0).sum()) == 4
