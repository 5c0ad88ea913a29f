"""Mixture-of-experts operators and weight-only FP4 products against plain 64-bit forms.

Tolerances follow from the arithmetic. u = 2^-24 is the float32 unit roundoff; the matrix cores
add with at most one ulp (2u) per product. A sum of m terms in any order is within m 2u of the sum
of magnitudes; the output's own rounding adds u (float32) or 2^-8 (bf16: 8 significant bits) of the value. Data of
small integers makes every sum exact, and then outputs are compared bit for bit.
"""
import numpy as np
import pytest
import torch

from oracle import formats as OF

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def gen(seed):
    return np.random.Generator(np.random.PCG64(seed))


def router_ids(r, tokens, topk, experts, drop):
    """Distinct choices where there are enough experts; dropped slots get ids on both sides of the range."""
    if topk <= experts:
        ids = np.argsort(r.random((tokens, experts)), axis=1)[:, :topk]
    else:
        ids = r.integers(0, experts, (tokens, topk))
    bad = r.choice(np.array([-1, experts, experts + 7, -2 ** 31, 2 ** 31 - 1]), size=ids.shape)
    return np.where(r.random(ids.shape) < drop, bad, ids).astype(np.int64)


def plain_sort(ids, experts):
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    order = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[order], np.arange(experts + 1))
    at = np.arange(len(flat))
    pos = np.empty(len(flat), np.int64)
    pos[order] = np.where(at < offsets[-1], at, ~at)
    return order, pos.reshape(ids.shape), offsets


def check_plan(plan, ids, experts, what):
    order, pos, offsets = plain_sort(ids, experts)
    assert np.array_equal(plan.offsets.cpu().numpy(), offsets), f"{what}: offsets"
    assert np.array_equal(plan.order.cpu().numpy(), order), f"{what}: order"
    assert np.array_equal(plan.pos.cpu().numpy(), pos), f"{what}: pos"


# ------------------------------------------------------------------ sort

@pytest.mark.parametrize("tokens,topk,experts,drop", [
    (1, 1, 1, 0.0), (1, 1, 1, 1.0), (1, 8, 256, 0.0), (16, 2, 8, 0.0), (63, 1, 2, 0.2), (65, 3, 3, 0.0), (1000, 4, 7, 0.3),
    (1024, 8, 64, 0.0), (1025, 8, 511, 0.1), (4096, 2, 512, 0.0), (512, 2, 1024, 0.1), (8192, 1, 8, 0.0),
    (8193, 1, 8, 0.0), (5000, 6, 160, 0.5), (30000, 8, 128, 0.02), (9000, 5, 1023, 0.0), (20000, 4, 3, 0.0),
    (700, 4, 300, 1.0),
])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(tokens, topk, experts, drop, dtype):
    import fp4_block_scaled_tensor_amd as fp4
    ids = router_ids(gen(tokens * 31 + experts), tokens, topk, experts, drop)
    dev = torch.from_numpy(ids).to(dtype).cuda()
    check_plan(fp4.expert_sort(dev, experts), ids, experts, "contiguous")
    wide = torch.full((tokens, topk + 3), -5, dtype=dtype, device="cuda")   # rows with a stride
    wide[:, 1:topk + 1] = dev
    check_plan(fp4.expert_sort(wide[:, 1:topk + 1], experts), ids, experts, "strided")


def test_sort_one_expert_takes_everything_and_large_int64_ids_drop():
    import fp4_block_scaled_tensor_amd as fp4
    for tokens in (300, 9000):
        ids = np.full((tokens, 2), 5, np.int64)
        check_plan(fp4.expert_sort(torch.from_numpy(ids).cuda(), 9), ids, 9, "one expert")
        ids[::3, 1] = 2 ** 32 + 5       # expert 5 in the low word only
        check_plan(fp4.expert_sort(torch.from_numpy(ids).cuda(), 9), ids, 9, "64-bit ids")


def test_empty_inputs():
    import fp4_block_scaled_tensor_amd as fp4
    plan = fp4.expert_sort(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 5)
    assert plan.offsets.cpu().tolist() == [0] * 6 and plan.order.numel() == 0
    x = torch.empty((0, 64), device="cuda")
    assert fp4.expert_gather(x, plan).shape == (0, 64) and fp4.expert_gather_grad(x, plan).shape == (0, 64)
    w = torch.empty((0, 2), device="cuda")
    assert fp4.expert_combine(x, w, plan).shape == (0, 64)
    dys, dw = fp4.expert_combine_grad(x, x, w, plan)
    assert dys.shape == (0, 64) and dw.shape == (0, 2)
    full = fp4.expert_sort(torch.zeros((3, 2), dtype=torch.int32, device="cuda"), 5)
    none = torch.empty((6, 0), device="cuda")
    _, dw = fp4.expert_combine_grad(none[:3], none, torch.ones((3, 2), device="cuda"), full)
    assert dw.cpu().tolist() == [[0.0, 0.0]] * 3


# ------------------------------------------------------------------ rows

def rows_case(seed, tokens, topk, experts, drop, hidden, dtype, layout):
    """ids, plan, and a maker of device matrices: contiguous, with padded rows, or off by one element."""
    import fp4_block_scaled_tensor_amd as fp4
    r = gen(seed)
    ids = router_ids(r, tokens, topk, experts, drop)
    plan = fp4.expert_sort(torch.from_numpy(ids).cuda(), experts)

    def make(rows, scale=1.0):
        v = torch.from_numpy((r.standard_normal((rows, hidden)) * scale).astype(np.float32)).to(dtype)
        if layout == "contiguous":
            return v.cuda()
        pad, off = {"padded": (16, 0), "shifted": (3, 1)}[layout]
        big = torch.full((rows, hidden + pad), float("nan"), dtype=dtype, device="cuda")
        big[:, off:off + hidden] = v.cuda()
        return big[:, off:off + hidden]
    return r, ids, plan, make


ROW_CASES = [
    (1, 1, 1, 0.0, 1), (1, 8, 16, 0.0, 8), (3, 2, 2, 0.0, 7), (33, 8, 64, 0.2, 4096), (257, 4, 9, 0.3, 1001),
    (130, 2, 8, 1.0, 72), (64, 6, 4, 0.0, 2048), (5, 3, 8, 0.3, 9000), (700, 1, 8, 0.1, 136), (40, 16, 32, 0.1, 520),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["contiguous", "padded", "shifted"])
@pytest.mark.parametrize("case", ROW_CASES, ids=str)
def test_rows(case, layout, dtype):
    import fp4_block_scaled_tensor_amd as fp4
    tokens, topk, experts, drop, hidden = case
    dt = DT[dtype]
    r, ids, plan, make = rows_case(hash(case) % 1000, tokens, topk, experts, drop, hidden, dt, layout)
    order, pos, offsets = plain_sort(ids, experts)
    kept, n = offsets[-1], tokens * topk
    x = make(tokens)
    xs = fp4.expert_gather(x, plan)
    want = torch.zeros((n, hidden), dtype=dt)
    want[:kept] = x.cpu()[order[:kept] // topk]
    assert torch.equal(xs.cpu(), want), "gather"

    ys = make(n)
    if kept < n:
        ys[kept:] = float("nan")                       # rows of dropped slots are never read
    y64 = ys.cpu().double().numpy()
    at = np.where(pos >= 0, pos, 0)
    live = (pos >= 0)[:, :, None]
    rows = np.where(live, y64[at], 0.0)
    got = fp4.expert_gather_grad(ys, plan).cpu().double().numpy()
    lim = topk * 2 * U * np.abs(rows).sum(1) * 1.01 + HALF_ULP[dt] * np.abs(rows.sum(1)) * 1.01
    assert (np.abs(got - rows.sum(1)) <= lim).all(), "gather_grad"

    w = r.standard_normal((tokens, topk)).astype(np.float32)
    wd = torch.from_numpy(w).cuda()
    wd[torch.from_numpy(pos < 0).cuda()] = float("nan")   # weights of dropped slots are never used
    if layout != "contiguous":
        wide = torch.full((tokens, topk + 5), float("nan"), device="cuda")
        wide[:, 2:topk + 2] = wd
        wd = wide[:, 2:topk + 2]
    got = fp4.expert_combine(ys, wd, plan).cpu().double().numpy()
    terms = rows * w[:, :, None].astype(np.float64)
    lim = (topk + 1) * 2 * U * np.abs(terms).sum(1) * 1.01 + HALF_ULP[dt] * np.abs(terms.sum(1)) * 1.01
    assert (np.abs(got - terms.sum(1)) <= lim).all(), "combine"

    dy = make(tokens, 1e-3)
    dys, dw = fp4.expert_combine_grad(dy, ys, wd, plan)
    dy64 = dy.cpu().double().numpy()
    want = np.zeros((n, hidden))
    s = order[:kept]
    want[:kept] = w.reshape(-1)[s].astype(np.float64)[:, None] * dy64[s // topk]
    got = dys.cpu().double().numpy()
    assert (np.abs(got - want) <= (HALF_ULP[dt] + U) * np.abs(want) * 1.01).all(), "dys"
    prod = rows * dy64[:, None, :]
    got = dw.cpu().double().numpy()
    assert (np.abs(got - prod.sum(2)) <= (hidden + 1) * U * np.abs(prod).sum(2) * 1.01).all(), "dw"
    assert (got[pos < 0] == 0).all(), "dw of dropped slots"


def test_row_values_pass_through():
    """Infinities, NaNs and signed zeros of kept rows reach the outputs; a token without kept slots gives zeros."""
    import fp4_block_scaled_tensor_amd as fp4
    ids = torch.tensor([[0, 1], [1, 5], [7, -1]], dtype=torch.int32, device="cuda")
    plan = fp4.expert_sort(ids, 4)
    x = torch.tensor([[float("inf"), -0.0], [float("nan"), 1.0], [2.0, 3.0]], device="cuda")
    xs = fp4.expert_gather(x, plan).cpu()
    assert xs[0].tolist() == xs[1].tolist() == [float("inf"), 0.0] and np.signbit(xs[0, 1].item())
    assert torch.isnan(xs[2, 0]) and xs[2, 1] == 1.0 and (xs[3:] == 0).all()
    y = fp4.expert_combine(xs.cuda(), torch.ones((3, 2), device="cuda"), plan).cpu()
    assert y[0].tolist() == [float("inf"), 0.0] and torch.isnan(y[1, 0]) and y[2].tolist() == [0.0, 0.0]


def test_row_gradients_match_differences():
    """With small integers every sum is exact, so the gradients equal differences of the forward: combine is
    linear in each input, and <dxs, gather(x)> = <gather_grad(dxs), x>."""
    import fp4_block_scaled_tensor_amd as fp4
    tokens, topk, experts, hidden = 37, 3, 5, 40
    r = gen(77)
    ids = router_ids(r, tokens, topk, experts, 0.2)
    plan = fp4.expert_sort(torch.from_numpy(ids).cuda(), experts)
    small = lambda *s: torch.from_numpy(r.integers(-4, 5, s).astype(np.float32)).cuda()   # noqa: E731
    ys, w, dy = small(tokens * topk, hidden), small(tokens, topk), small(tokens, hidden)
    dys, dw = fp4.expert_combine_grad(dy, ys, w, plan)
    loss = lambda a, b: (fp4.expert_combine(a, b, plan).double() * dy.double()).sum().item()   # noqa: E731
    base = loss(ys, w)
    for t, j in [(0, 0), (5, 1), (36, 2), (20, 0)]:
        w2 = w.clone()
        w2[t, j] += 1
        assert loss(ys, w2) - base == dw[t, j].item()
    for p, h in [(0, 0), (50, 39), (110, 7), (81, 20)]:
        y2 = ys.clone()
        y2[p, h] += 1
        assert loss(y2, w) - base == dys[p, h].item()
    x, dxs = small(tokens, hidden), small(tokens * topk, hidden)
    lhs = (dxs.double() * fp4.expert_gather(x, plan).double()).sum()
    assert lhs == (fp4.expert_gather_grad(dxs, plan).double() * x.double()).sum()


def test_rows_skip_positions_out_of_range():
    """Positions outside the tensor are skipped by the kernels' own bounds checks."""
    import fp4_block_scaled_tensor_amd as fp4
    pos = torch.tensor([[0, 99], [-101, 2]], dtype=torch.int32, device="cuda")
    plan = fp4.ExpertPlan(torch.zeros(4, dtype=torch.int32, device="cuda"), pos, torch.zeros(3, dtype=torch.int32,
                          device="cuda"), 2, 2, 2)
    x = torch.arange(1.0, 17.0, device="cuda").view(2, 8)
    out = torch.full((4, 8), -1.0, device="cuda")
    fp4.expert_gather(x, plan, out=out)
    assert torch.equal(out[0], x[0]) and torch.equal(out[2], x[1]) and (out[1] == -1).all() and (out[3] == -1).all()
    ys = torch.arange(1.0, 33.0, device="cuda").view(4, 8)
    assert torch.equal(fp4.expert_gather_grad(ys, plan), ys[[0, 2]])
    _, dw = fp4.expert_combine_grad(x, ys, torch.ones((2, 2), device="cuda"), plan)
    assert dw[0, 1] == 0 and dw[1, 0] == 0 and dw[1, 1] == (x[1] * ys[2]).sum()


def test_rows_past_32_bit_offsets():
    """Expert rows of more than 2^32 bytes and 2^31 elements."""
    import fp4_block_scaled_tensor_amd as fp4
    tokens, topk, hidden = 140000, 2, 8192
    ids = torch.zeros((tokens, topk), dtype=torch.int32, device="cuda")
    ids[:, 1] = 1
    plan = fp4.expert_sort(ids, 2)
    x = torch.zeros((tokens, hidden), dtype=torch.bfloat16, device="cuda")
    x[:, :8] = torch.arange(tokens, device="cuda")[:, None] % 251 + torch.arange(8, device="cuda")
    xs = fp4.expert_gather(x, plan)
    assert torch.equal(xs[:tokens], x) and torch.equal(xs[tokens:], x)
    y = fp4.expert_combine(xs, torch.full((tokens, topk), 0.5, device="cuda"), plan)
    assert torch.equal(y, x)


# ------------------------------------------------------------------ products

LAYOUTS = {"1d": 0, "2d": 1, "2dT": 2}
FMTS = {"ue5m3": OF.UE5M3, "e4m3": OF.E4M3, "e8m0": OF.E8M0}


def random_weight(r, n, k, fmt, block, layout, g=1.0, ones=False, spread=2):
    """A weight of random codes as a device QTensor and its float64 values [n, k]."""
    import fp4_block_scaled_tensor_amd as fp4
    f = FMTS[fmt]
    codes = r.integers(0, 16, (n, k)).astype(np.uint8)
    shape = {"1d": (n, k // block), "2d": (n // 16, k // 16), "2dT": (k // 16, n // 16)}[layout]
    one = OF.SCALE_ONE_CODE[f]
    step = 1 if f == OF.E8M0 else 8
    sc = np.full(shape, one) if ones else one + r.integers(-spread * step, spread * step + 1, shape)
    sc = sc.astype(np.uint8)
    return weight_from(codes, sc, f, block, layout, g)


def weight_from(codes, sc, f, block, layout, g, g_stripe=0):
    import fp4_block_scaled_tensor_amd as fp4
    n, k = codes.shape
    s64 = OF.SCALE_VALUES[f][sc]
    if layout == "2dT":
        s64 = s64.T
    if layout != "1d":
        s64 = np.repeat(s64, 16, axis=0)
    w64 = OF.E2M1_VALUES[codes] * np.repeat(s64, block, axis=1)
    gt = torch.tensor(np.atleast_1d(np.float32(g)), device="cuda")
    q = torch.from_numpy(codes[:, 0::2] | (codes[:, 1::2] << 4)).cuda()
    return fp4.QTensor(q, torch.from_numpy(sc).cuda(), gt, f, block, LAYOUTS[layout], n, k, g_stripe), w64


def close(got, x64, w64, g, out_dt, what):
    """got within the bound of x . w^T * g: K products and one multiply by g, then the output's rounding."""
    ref = (x64 @ w64.T) * g
    mag = (np.abs(x64) @ np.abs(w64).T) * np.abs(g)
    lim = ((x64.shape[1] + 1) * 2 * U * mag + HALF_ULP[out_dt] * np.abs(ref)) * 1.01
    bad = np.abs(got.cpu().double().numpy() - ref) > lim
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, first at {tuple(np.argwhere(bad)[0])}"


WEIGHTS = [("ue5m3", 16, "1d"), ("ue5m3", 16, "2d"), ("ue5m3", 16, "2dT"), ("ue5m3", 32, "1d"), ("e4m3", 16, "1d"),
           ("e4m3", 16, "2dT"), ("e4m3", 32, "1d"), ("e8m0", 32, "1d")]
SIZES = [(1, 16, 64), (1, 1000, 4096), (2, 33, 192), (7, 48, 1088), (16, 272, 256), (17, 100, 320), (33, 512, 576),
         (64, 80, 2048), (65, 144, 448), (100, 1000, 832), (130, 304, 512), (256, 256, 256), (300, 520, 1600),
         (515, 777, 640)]


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("fmt,block,layout", WEIGHTS)
def test_linear(fmt, block, layout, dtype, out):
    import fp4_block_scaled_tensor_amd as fp4
    for i, (m, n, k) in enumerate(SIZES):
        if layout != "1d":
            n = -(-n // 16) * 16
        r = gen(1000 + i)
        w, w64 = random_weight(r, n, k, fmt, block, layout, g=0.37)
        x = torch.from_numpy(r.standard_normal((m, k)).astype(np.float32)).to(DT[dtype]).cuda()
        y = fp4.linear(x, w, out_dtype=DT[out])
        assert y.dtype == DT[out]
        close(y, x.cpu().double().numpy(), w64, float(np.float32(0.37)), DT[out], f"{m}x{n}x{k}")


# Sizes that take every kernel shape: few rows with one, two and four products to a fragment and 4, 8 and 16 rows
# at a time; tiles of 32 to 256 rows, with and without a split K. K = 192 and 320 end half way into a turn.
# (With a split K these are 32-row tiles; test_gpu_wlinear_split.py takes the taller ones.)
SHAPES = [(1, 8208, 192), (3, 16400, 192), (7, 8208, 320), (8, 16400, 128), (12, 16400, 192), (16, 8208, 192),
          (20, 4112, 1088), (100, 32784, 192), (90, 16400, 320), (50, 65616, 64), (2045, 6160, 192), (1030, 8208, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,block,layout", [("ue5m3", 16, "1d"), ("e4m3", 16, "2dT"), ("e4m3", 32, "1d"), ("e8m0", 32, "1d")])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_every_shape(shape, fmt, block, layout, dtype):
    """Exact on integers (quantum 2^-6, sums below 2^18), in float64 on the device."""
    import fp4_block_scaled_tensor_amd as fp4
    m, n, k = shape
    r = gen(m + n)
    w, _ = random_weight(r, n, k, fmt, block, layout, spread=1)
    x = torch.from_numpy(r.integers(-8, 9, (m, k)).astype(np.float32)).to(DT[dtype]).cuda()
    y = fp4.linear(x, w, out_dtype=torch.float32)
    want = x.double() @ fp4.dequantize(w).double().t().contiguous()
    assert torch.equal(y.double(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,block,layout", WEIGHTS)
def test_linear_exact_on_integers(fmt, block, layout, dtype):
    """Integers whose sums stay below 2^24 quanta: every product and sum is exact, so outputs match bit for bit."""
    import fp4_block_scaled_tensor_amd as fp4
    for i, (m, n, k) in enumerate(SIZES):
        if layout != "1d":
            n = -(-n // 16) * 16
        r = gen(2000 + i)
        w, w64 = random_weight(r, n, k, fmt, block, layout, spread=1)
        x64 = r.integers(-8, 9, (m, k)).astype(np.float64)
        x = torch.from_numpy(x64).to(DT[dtype]).cuda()
        y = fp4.linear(x, w, out_dtype=torch.float32)
        # quantum 2^-6 (E2M1 halves, scale eighths and halves); sums below 8 * 12 * 1088 < 2^18
        assert np.array_equal(y.cpu().double().numpy(), x64 @ w64.T), f"{m}x{n}x{k}"


def test_linear_keeps_all_bits_of_float32():
    """A one-hot float32 row with 24 significant bits times a weight of 1: the three bf16 parts carry every bit."""
    import fp4_block_scaled_tensor_amd as fp4
    k, n, f = 128, 48, OF.UE5M3
    w, _ = weight_from(np.full((n, k), 2, np.uint8), np.full((n, k // 16), OF.SCALE_ONE_CODE[f], np.uint8), f, 16, "1d", 1.0)
    vals = np.array([16777215.0, -8388609.0, 1 + 2.0 ** -23, 3.4028235e38, -1.1754944e-20, 0.1, np.pi, 1e-30], np.float32)
    for m in (8, 96, 300):
        x = np.zeros((m, k), np.float32)
        for i in range(m):
            x[i, (i * 37) % k] = vals[i % 8]
        y = fp4.linear(torch.from_numpy(x).cuda(), w).cpu().numpy()
        assert np.array_equal(y, np.repeat(x.sum(1)[:, None], n, 1)), m


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [3, 40, 280])
def test_linear_infinities_and_nans(m, dtype):
    """An infinite or NaN activation reaches its own row's outputs only, as in the plain product."""
    import fp4_block_scaled_tensor_amd as fp4
    r = gen(5)
    k, n = 192, 80
    w, w64 = random_weight(r, n, k, "ue5m3", 16, "1d")
    w64[w64 == 0] = 0.0
    x = torch.from_numpy(r.standard_normal((m, k)).astype(np.float32)).to(DT[dtype])
    x[0, 5], x[1, 190], x[2, 64] = float("inf"), float("-inf"), float("nan")
    got = fp4.linear(x.cuda(), w, out_dtype=torch.float32).cpu().double().numpy()
    with np.errstate(invalid="ignore"):
        want = x.double().numpy() @ w64.T
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isposinf(got), np.isposinf(want))
    assert np.isnan(got[2]).all() and np.isfinite(got[3:]).all()


@pytest.mark.parametrize("m", [1, 300])
def test_linear_every_scale_code(m):
    """Every scale code of each format (E8M0: up to 2^121), one weight row per code; products past the float32 range
    are infinite."""
    import fp4_block_scaled_tensor_amd as fp4
    for fmt, f in FMTS.items():
        codes_s = np.arange(len(OF.SCALE_VALUES[f]) if f != OF.E8M0 else 249)   # 6 * 2^121 and below stay finite
        block = 32 if f == OF.E8M0 else 16
        n = len(codes_s)
        sc = np.repeat(codes_s[:, None], 64 // block, 1).astype(np.uint8)
        w, w64 = weight_from(np.full((n, 64), 3, np.uint8), sc, f, block, "1d", 1.0)    # 1.5 * S
        x = np.zeros((m, 64), np.float32)
        x[:, 17] = 2.0 if f != OF.E8M0 else 2.0 ** 20
        y = fp4.linear(torch.from_numpy(x).cuda(), w).cpu().double().numpy()
        with np.errstate(over="ignore"):
            want = (x[:1].astype(np.float64) @ w64.T).astype(np.float32)
        assert np.array_equal(y, np.repeat(want, m, 0)), fmt


def test_linear_g_forms_strides_and_alignment():
    """g per stripe or absent, activations with a row stride, outputs into rows of any stride, guarded."""
    import fp4_block_scaled_tensor_amd as fp4
    r = gen(9)
    for m in (5, 90, 400):
        n, k = 200, 320
        codes = r.integers(0, 16, (n, k)).astype(np.uint8)
        sc = np.full((n, k // 16), OF.SCALE_ONE_CODE[OF.E4M3], np.uint8)
        g = (r.random(-(-n // 32)) + 0.5).astype(np.float32)
        w, w64 = weight_from(codes, sc, OF.E4M3, 16, "1d", g, g_stripe=32)
        big = torch.full((m, k + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
        x = big[:, 8:8 + k]
        x.copy_(torch.from_numpy(r.standard_normal((m, k))).to(torch.bfloat16))
        out = torch.full((m, n + 7), -77.0, dtype=torch.bfloat16, device="cuda")
        fp4.linear(x, w, out=out[:, 3:3 + n])
        close(out[:, 3:3 + n], x.cpu().double().numpy(), w64, np.repeat(g, 32)[:n].astype(np.float64)[None],
              torch.bfloat16, "stripes")
        assert (out[:, :3] == -77).all() and (out[:, 3 + n:] == -77).all()


def test_linear_transposed_view_is_the_gradient():
    """One TILE2D quantization: linear with the transposed operand is the gradient of linear with the forward one
    (exact on integers: <dy, x W^T> = <dy W, x>), and a unit change of x changes y by the weight's column."""
    import fp4_block_scaled_tensor_amd as fp4
    r = gen(12)
    n, k = 192, 320
    wt = torch.from_numpy(r.standard_normal((n, k)).astype(np.float32)).cuda()
    fwd, bwd = fp4.quantize(wt, fp4.UE5M3, 16, fp4.TILE2D, amax=fp4.tensor_amax(wt))
    w64 = fp4.dequantize(fwd).double().cpu().numpy()
    for m in (4, 80, 270):
        x64, dy64 = r.integers(-3, 4, (m, k)).astype(np.float64), r.integers(-3, 4, (m, n)).astype(np.float64)
        x, dy = (torch.from_numpy(v).to(torch.bfloat16).cuda() for v in (x64, dy64))
        dx = fp4.linear(dy, bwd, out_dtype=torch.float32)
        close(dx, dy64, w64.T, 1.0, torch.float32, "dx")
        y = fp4.linear(x, fwd, out_dtype=torch.float32)
        lhs, rhs = (y.double().cpu().numpy() * dy64).sum(), (dx.double().cpu().numpy() * x64).sum()
        # both sides sum m n k products, each within (K + 1) 2u
        lim = (max(n, k) + 1) * 2 * U * (np.abs(dy64) @ np.abs(w64) * np.abs(x64)).sum() * 2
        assert abs(lhs - rhs) <= lim
        x2 = x.clone()
        x2[1, 7] += 1
        diff = (fp4.linear(x2, fwd, out_dtype=torch.float32) - y).double().cpu().numpy()
        assert (diff[0] == 0).all() and (diff[2:] == 0).all()
        lim = 2 * (k + 1) * 2 * U * (np.abs(x64[1:2]) + (np.arange(k) == 7)) @ np.abs(w64).T
        assert (np.abs(diff[1] - w64[:, 7]) <= lim[0]).all()


EXPERT_CASES = [
    # rows of each expert, dropped rows
    ([1], 0), ([0, 0, 3, 0], 0), ([2, 1, 0, 5, 4, 0, 1, 1], 2), ([40, 0, 7, 129], 5), ([0, 300, 1, 17], 0),
    ([64] * 6, 0), ([0, 0], 9), ([0] * 30 + [200] + [1] * 33, 4), ([1] * 70 + [30], 0), ([3] * 130 + [0], 1), ([513, 2, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0], 1), ([256, 255, 257], 3),
]


@pytest.mark.parametrize("fmt,block,layout", [("ue5m3", 16, "1d"), ("ue5m3", 16, "2d"), ("e4m3", 16, "2dT"),
                                              ("e4m3", 32, "1d"), ("e8m0", 32, "1d")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_expert_linear(fmt, block, layout, dtype):
    import fp4_block_scaled_tensor_amd as fp4
    for i, (counts, dropped) in enumerate(EXPERT_CASES):
        r = gen(3000 + i)
        k, n = [64, 320, 576][i % 3], [48, 208, 304][(i + 1) % 3] + (0 if layout != "1d" else 5)
        pairs = [random_weight(r, n, k, fmt, block, layout, g=0.5 + e) for e in range(len(counts))]
        stack = fp4.stack_experts([p[0] for p in pairs])
        ends = np.concatenate([[0], np.cumsum(counts)])
        rows = int(ends[-1]) + dropped
        x = torch.from_numpy(r.standard_normal((rows, k)).astype(np.float32)).to(DT[dtype]).cuda()
        x[int(ends[-1]):] = float("nan")                       # rows of dropped slots are not used
        offsets = torch.from_numpy(ends.astype(np.int32)).cuda()
        out = torch.full((rows, n), float("nan"), dtype=torch.float32, device="cuda")
        fp4.expert_linear(x, stack, offsets, out=out)
        assert (out[int(ends[-1]):] == 0).all(), "dropped rows"
        for e in range(len(counts)):
            if counts[e]:
                a, b = int(ends[e]), int(ends[e + 1])
                close(out[a:b], x[a:b].cpu().double().numpy(), pairs[e][1], 0.5 + e, torch.float32, f"case {i} expert {e}")


@pytest.mark.parametrize("fmt,block,layout", [("ue5m3", 16, "1d"), ("e4m3", 16, "2dT"), ("e8m0", 32, "1d")])
@pytest.mark.parametrize("counts,n", [([1000, 1, 0, 1044], 6160), ([2, 0, 1, 0, 3], 8208), ([40, 30, 0, 50], 16400)])
def test_expert_linear_large(counts, n, fmt, block, layout):
    """Tall tiles and wide weights over experts, exact on integers."""
    import fp4_block_scaled_tensor_amd as fp4
    r, k = gen(n), 192
    ws = [random_weight(r, n, k, fmt, block, layout, spread=1)[0] for _ in counts]
    ends = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x = torch.from_numpy(r.integers(-8, 9, (int(ends[-1]) + 3, k)).astype(np.float32)).to(torch.bfloat16).cuda()
    y = fp4.expert_linear(x, fp4.stack_experts(ws), torch.from_numpy(ends).cuda(), out_dtype=torch.float32)
    assert (y[int(ends[-1]):] == 0).all()
    for e, w in enumerate(ws):
        a, b = int(ends[e]), int(ends[e + 1])
        assert torch.equal(y[a:b].double(), x[a:b].double() @ fp4.dequantize(w).double().t().contiguous()), e


def test_expert_linear_bad_offsets_stay_in_bounds():
    """Offsets outside the tensor are clamped by the kernel: nothing outside the rows is touched."""
    import fp4_block_scaled_tensor_amd as fp4
    r = gen(31)
    pairs = [random_weight(r, 32, 64, "e8m0", 32, "1d") for _ in range(3)]
    stack = fp4.stack_experts([p[0] for p in pairs])
    x = torch.from_numpy(r.standard_normal((20, 64)).astype(np.float32)).to(torch.bfloat16).cuda()
    guard = torch.full((40, 32), -3.0, device="cuda")
    offsets = torch.tensor([-5, 4, 1000, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    fp4.expert_linear(x, stack, offsets, out=guard[10:30])
    assert (guard[:10] == -3).all() and (guard[30:] == -3).all()
    close(guard[10:14], x[:4].cpu().double().numpy(), pairs[0][1], 1.0, torch.float32, "expert 0")
    close(guard[14:30], x[4:].cpu().double().numpy(), pairs[1][1], 1.0, torch.float32, "expert 1")


def test_expert_weights_past_32_bit_offsets():
    """A stack of more than 2^32 payload bytes; only its last experts have rows."""
    import fp4_block_scaled_tensor_amd as fp4
    n = k = 8192
    experts = 140
    q = torch.zeros((experts, n, k // 2), dtype=torch.uint8, device="cuda")
    s = torch.full((experts, n, k // 32), 127, dtype=torch.uint8, device="cuda")
    q[-1, :, 0] = 2                  # weight 1 at k = 0
    q[-2, :, 0] = 4                  # weight 2
    stack = fp4.ExpertWeights(q, s, torch.ones((experts, 1), device="cuda"), fp4.E8M0, 32, fp4.FP4_SCALES_1D, n, k)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    for rows in (8, 40000):
        offsets[-2], offsets[-1] = rows // 2, rows
        x = torch.zeros((rows, k), dtype=torch.bfloat16, device="cuda")
        x[:, 0] = torch.arange(rows, device="cuda") % 200 + 1
        y = fp4.expert_linear(x, stack, offsets)
        assert torch.equal(y[:rows // 2], (2 * x[:rows // 2, :1]).expand(-1, n))
        assert torch.equal(y[rows // 2:], x[rows // 2:, :1].expand(-1, n))


# ------------------------------------------------------------------ streams, graphs, determinism

def layer(fp4, x, ids, w, up, down):
    plan = fp4.expert_sort(ids, up.n_experts)
    h = fp4.expert_linear(fp4.expert_gather(x, plan), up, plan)
    h = torch.nn.functional.silu(h.float()).to(h.dtype)
    ys = fp4.expert_linear(h, down, plan)
    y = fp4.expert_combine(ys, w, plan)
    return [y, *fp4.expert_combine_grad(y, ys, w, plan), fp4.expert_gather_grad(ys, plan)]


@pytest.mark.parametrize("tokens,topk", [(5, 2), (600, 2), (3000, 4)])
def test_layer_on_a_stream_in_a_graph_and_again(tokens, topk):
    """The operators together: on a side stream, captured in a graph and replayed with eager work between, and
    again eagerly, always with the same bits."""
    import fp4_block_scaled_tensor_amd as fp4
    r = gen(61)
    experts, hidden, ffn = 6, 256, 448
    up = fp4.stack_experts([random_weight(r, ffn, hidden, "ue5m3", 16, "1d", g=0.1)[0] for _ in range(experts)])
    down = fp4.stack_experts([random_weight(r, hidden, ffn, "e8m0", 32, "1d", g=0.1)[0] for _ in range(experts)])
    x = torch.from_numpy(r.standard_normal((tokens, hidden)).astype(np.float32)).to(torch.bfloat16).cuda()
    ids = torch.from_numpy(router_ids(r, tokens, topk, experts, 0.1)).cuda()
    w = torch.from_numpy(r.random((tokens, topk)).astype(np.float32)).cuda()
    want = [t.clone() for t in layer(fp4, x, ids, w, up, down)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer(fp4, x, ids, w, up, down)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    bits = lambda t: t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)   # noqa: E731
    for a, b in zip(got, want):
        assert torch.equal(bits(a), bits(b)), "side stream"
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = layer(fp4, x, ids, w, up, down)
    for rep in range(3):
        for t in kept:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(kept, want):
            assert torch.equal(bits(a), bits(b)), f"replay {rep}"
        for a, b in zip(layer(fp4, x, ids, w, up, down), want):
            assert torch.equal(bits(a), bits(b)), f"eager {rep}"
