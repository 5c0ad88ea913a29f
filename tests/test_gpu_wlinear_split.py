"""Weight-only products whose K is split over workgroups: the documented order of the arithmetic (all of the
sum, then g), and exact sums in every tile height."""
import numpy as np
import pytest
import torch

from oracle import formats as OF

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def ones_weight(n, k, g, g_stripe=0):
    import fp4_block_scaled_tensor_amd as fp4
    q = torch.full((n, k // 2), 0x22, dtype=torch.uint8, device="cuda")
    s = torch.full((n, k // 16), int(OF.SCALE_ONE_CODE[OF.UE5M3]), dtype=torch.uint8, device="cuda")
    return fp4.QTensor(q, s, torch.tensor(np.atleast_1d(np.float32(g)), device="cuda"), fp4.UE5M3, 16,
                       fp4.FP4_SCALES_1D, n, k, g_stripe)


def cancelling_rows(m, k, dt):
    """Row r sums to r + 1; its first and last elements, far apart along K, cancel."""
    x = np.zeros((m, k), np.float32)
    x[:, 0], x[:, -1], x[:, 1] = 1024, -1024, np.arange(1, m + 1)
    return torch.from_numpy(x).to(dt).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("n,stripe", [(48, 0), (45, 0), (48, 16), (45, 32)])
def test_g_multiplies_the_whole_sum(n, stripe, out, dtype):
    """g * 1024 is infinite, g times the sum is not: a part of K multiplied by g before the parts are joined would
    leave infinity minus infinity. (r + 1) * g is exact in float32."""
    import fp4_block_scaled_tensor_amd as fp4
    m, k = 40, 4096
    g = np.float32(2.0 ** 118) * (1 + np.arange(-(-n // stripe) if stripe else 1, dtype=np.float32) / 4)
    y = fp4.linear(cancelling_rows(m, k, DT[dtype]), ones_weight(n, k, g, stripe), out_dtype=DT[out])
    want = np.arange(1, m + 1, dtype=np.float32)[:, None] * (np.repeat(g, stripe)[:n] if stripe else np.repeat(g, n))
    assert torch.equal(y.cpu(), torch.from_numpy(want).to(DT[out]))


@pytest.mark.parametrize("stripe", [0, 32])
@pytest.mark.parametrize("n", [64, 37])
def test_each_rows_expert_gives_its_g(n, stripe):
    """The same for rows in expert order: empty experts (whose g is NaN) first, between and last, dropped rows zero."""
    import fp4_block_scaled_tensor_amd as fp4
    k, counts, dropped = 2048, [0, 20, 0, 0, 41, 1, 0], 3
    per = -(-n // stripe) if stripe else 1
    g = [np.float32(2.0 ** 118) * (1 + (e + np.arange(per)) % 4 / 4) if c else np.full(per, np.nan) for e, c in enumerate(counts)]
    stack = fp4.stack_experts([ones_weight(n, k, v, stripe) for v in g])
    ends = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(ends[-1]) + dropped
    x = cancelling_rows(rows * 2, k, torch.float32)[:rows]
    x = torch.cat([x, torch.zeros((60, k), device="cuda")])       # more dropped rows: past 16 rows to an expert
    y = fp4.expert_linear(x, stack, torch.from_numpy(ends).cuda()).cpu().numpy()
    want = np.zeros((rows + 60, n), np.float32)
    for e, c in enumerate(counts):
        v = np.float32(g[e])
        for r in range(ends[e], ends[e] + c):
            want[r] = np.float32(r + 1) * (np.repeat(v, stripe)[:n] if stripe else np.repeat(v, n))
    assert np.array_equal(y, want)


# Sizes whose K is split, and the tile heights they take on 256 compute units: 32, 64, 96, 128 and 256 rows. 19
# steps of K: the parts begin at even and at odd turns of two steps, and the last turn is half a turn.
SPLIT = [(77, 1024), (77, 6144), (150, 6144), (200, 6144), (200, 12288)]
SPLIT_EXPERTS = [([30, 0, 17, 30], 1024, 0), ([1, 60, 0, 9], 4096, 7), ([97, 0, 30, 20], 4096, 3), ([129, 1, 0, 64], 4096, 6),
                 ([700, 300, 1, 490], 2048, 9)]
K = 1216


def workspace_slices(rows, w, experts):
    """Parts of K that the call's workspace has room for (bf16 rows: nothing else is in it)."""
    from fp4_block_scaled_tensor_amd import experts as E
    nb = E._linear_workspace(rows, 0, w.fmt, w.block, w.layout, w.g_stripe, w.rows, w.k, experts)
    return nb // (4 * rows * w.rows)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,block,layout", [("ue5m3", 16, "1d"), ("e4m3", 16, "2dT"), ("e8m0", 32, "1d")])
@pytest.mark.parametrize("m,n", SPLIT)
def test_split_k_in_every_tile_height(m, n, fmt, block, layout, dtype):
    """Exact on integers (quantum 2^-6, sums below 8 * 12 * 1216 < 2^17): equal to float64 bit for bit."""
    import fp4_block_scaled_tensor_amd as fp4
    from test_gpu_experts import gen, random_weight
    r = gen(m + n)
    n -= 9 if fmt == "e8m0" else 0                       # rows of y without 16-byte alignment
    w, _ = random_weight(r, n, K, fmt, block, layout, spread=1)
    assert workspace_slices(m, w, 0) > 1
    x = torch.from_numpy(r.integers(-8, 9, (m, K)).astype(np.float32)).to(DT[dtype]).cuda()
    y = fp4.linear(x, w, out_dtype=torch.float32)
    assert torch.equal(y.double(), x.double() @ fp4.dequantize(w).double().t().contiguous())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,block,layout", [("ue5m3", 16, "1d"), ("e8m0", 32, "1d")])
@pytest.mark.parametrize("counts,n,dropped", SPLIT_EXPERTS)
def test_split_k_over_experts(counts, n, dropped, fmt, block, layout, dtype):
    import fp4_block_scaled_tensor_amd as fp4
    from test_gpu_experts import gen, random_weight
    r = gen(sum(counts) + n)
    pairs = [random_weight(r, n, K, fmt, block, layout, g=2.0 ** e, spread=1) for e in range(len(counts))]
    stack = fp4.stack_experts([p[0] for p in pairs])
    ends = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(ends[-1]) + dropped
    assert workspace_slices(rows, stack, len(counts)) > 1
    x = torch.from_numpy(r.integers(-8, 9, (rows, K)).astype(np.float32)).to(DT[dtype]).cuda()
    x[int(ends[-1]):] = float("nan")                     # rows of dropped slots are not used
    y = fp4.expert_linear(x, stack, torch.from_numpy(ends).cuda(), out_dtype=torch.float32)
    assert (y[int(ends[-1]):] == 0).all()
    for e, (_, w64) in enumerate(pairs):
        a, b = int(ends[e]), int(ends[e + 1])
        if a < b:
            want = (x[a:b].double() @ torch.from_numpy(w64.T.copy()).cuda()) * 2.0 ** e
            assert torch.equal(y[a:b].double(), want), e


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("n", [64, 19, 1])
@pytest.mark.parametrize("experts", [1, 2, 62, 63, 64, 65, 130])
def test_g_of_many_experts(experts, n, out):
    """Each row gets its own expert's g, rows of empty and of one-row experts next to each other; exact on integers."""
    import fp4_block_scaled_tensor_amd as fp4
    from test_gpu_experts import gen
    r, k = gen(experts), 512
    counts = r.choice([0, 1, 2, 40], experts, p=[0.2, 0.2, 0.2, 0.4])
    counts[-1] = 40
    ends = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = max(int(ends[-1]) + 5, 17 * experts)
    g = 2.0 ** np.arange(-(experts // 2), experts - experts // 2).clip(-30, 30)
    w = ones_weight(n, k, 1.0)
    stack = fp4.ExpertWeights(w.q.expand(experts, -1, -1).contiguous(), w.s.expand(experts, -1, -1).contiguous(),
                              torch.tensor(g, dtype=torch.float32, device="cuda").view(-1, 1), w.fmt, 16, w.layout, n, k)
    assert workspace_slices(rows, stack, experts) > 1
    x64 = r.integers(-4, 5, (rows, k)).astype(np.float64)
    y = fp4.expert_linear(torch.from_numpy(x64).to(torch.bfloat16).cuda(), stack, torch.from_numpy(ends).cuda(),
                          out_dtype=DT[out])
    scale = np.concatenate([np.repeat(g, counts), np.zeros(rows - int(ends[-1]))])
    want = np.repeat((x64.sum(1) * scale)[:, None], n, 1).astype(np.float32)
    assert torch.equal(y.cpu(), torch.from_numpy(want).to(DT[out]))
