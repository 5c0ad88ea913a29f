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
