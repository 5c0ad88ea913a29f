"""The ends of the range of weight-only products: the largest power-of-two scales and the smallest float32
activations. One product to an output, so every finite value below is exact."""
import numpy as np
import pytest
import torch

from oracle import formats as OF

pytestmark = pytest.mark.gpu


def one_product_weight(codes, scale_codes, k=64, at=17):
    """Row n holds codes[n] times 2^(scale_codes[n] - 127) in column `at`, zeros elsewhere."""
    import fp4_block_scaled_tensor_amd as fp4
    n = len(codes)
    nibbles = np.zeros((n, k), np.uint8)
    nibbles[:, at] = codes
    q = torch.from_numpy(nibbles[:, 0::2] | (nibbles[:, 1::2] << 4)).cuda()
    s = torch.from_numpy(np.repeat(np.asarray(scale_codes, np.uint8)[:, None], k // 32, 1).copy()).cuda()
    return fp4.QTensor(q, s, torch.ones(1, device="cuda"), fp4.E8M0, 32, fp4.FP4_SCALES_1D, n, k)


def rows_of(values, m, k=64, at=17):
    x = np.zeros((m, k), np.float32)
    x[:, at] = np.resize(np.asarray(values, np.float32), m)
    return x


@pytest.mark.parametrize("m", [3, 40, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_largest_power_of_two_scales(m, dtype):
    """Codes up to 252 are exact with every E2M1 value; 253 and 254 where the weight stays below 2^128, from which on
    it is infinite (with float32 activations, whose lower parts are zero, infinite or NaN)."""
    import fp4_block_scaled_tensor_amd as fp4
    codes, scales = (v.reshape(-1) for v in np.meshgrid(np.arange(16), np.arange(247, 255)))
    w64 = OF.E2M1_VALUES[codes] * 2.0 ** (scales.astype(np.float64) - 127)
    x = rows_of([2.0 ** -10, -1.5 * 2.0 ** -60, 1.0, 2.0 ** -126], m)
    x[:, 17] = np.where(np.arange(m) % 4 == 2, 2.0 ** -2, x[:, 17])       # 6 * 2^125 * 2^-2 is finite
    y = fp4.linear(torch.from_numpy(x).to(dtype).cuda(), one_product_weight(codes, scales), out_dtype=torch.float32)
    y = y.cpu().numpy()
    finite = np.abs(w64) < 2.0 ** 128
    assert finite[scales <= 252].all() and (~finite).sum() == 2 * (2 + 4)
    want = x[:, 17].astype(np.float64)[:, None] * w64[None]
    assert np.array_equal(y[:, finite], want[:, finite])
    past = y[:, ~finite]
    if dtype is torch.bfloat16:
        assert np.isinf(past).all() and np.array_equal(np.sign(past), np.sign(want[:, ~finite]))
    else:
        assert not np.isfinite(past).any()


@pytest.mark.parametrize("m", [3, 40, 300])
def test_smallest_float32_activations(m):
    """The three parts add up to x exactly from 2^-110 on; from 2^-126 to there within 2^-133."""
    import fp4_block_scaled_tensor_amd as fp4
    r = np.random.Generator(np.random.PCG64(m))
    mantissa = 1 + r.integers(0, 2 ** 23, m) / 2.0 ** 23
    mantissa[0] = 2 - 2.0 ** -23                                            # all 24 bits
    for e in (-100, -109, -110, -111, -118, -125, -126):
        x = rows_of(mantissa * 2.0 ** e, m)
        y = fp4.linear(torch.from_numpy(x).cuda(), one_product_weight([2] * 24, [127] * 24)).cpu().numpy()
        err = np.abs(y.astype(np.float64) - x[:, 17].astype(np.float64)[:, None])
        assert (err == 0).all() if e >= -110 else (err < 2.0 ** -133).all(), e


@pytest.mark.parametrize("dtype,n", [(torch.float32, 2 ** 29 + 16), (torch.bfloat16, 2 ** 30 + 16)])
@pytest.mark.parametrize("m", [1, 17])
def test_more_weight_rows_than_one_launch_of_the_rows_form_holds(m, dtype, n):
    """A grid holds less than 2^32 threads: from 2^29 weight rows on (2^30 for bf16 activations) one row of
    activations needs another form than few rows usually take."""
    import fp4_block_scaled_tensor_amd as fp4
    k = 64
    q = torch.zeros((n, k // 2), dtype=torch.uint8, device="cuda")
    rows = [0, 255, 256, 2 ** 28 + 1, n - 17, n - 1]
    for i, row in enumerate(rows):
        q[row, 3] = 2 + i                                    # E2M1 code 2 + i at k = 6
    w = fp4.QTensor(q, torch.full((n, 2), 127, dtype=torch.uint8, device="cuda"), torch.ones(1, device="cuda"), fp4.E8M0,
                    32, fp4.FP4_SCALES_1D, n, k)
    x = torch.zeros((m, k), dtype=dtype, device="cuda")
    x[:, 6] = torch.arange(1, m + 1, device="cuda")
    y = fp4.linear(x, w, out_dtype=torch.bfloat16)
    want = torch.arange(1, m + 1)[:, None] * torch.from_numpy(OF.E2M1_VALUES[[2 + i for i in range(6)]])
    assert torch.equal(y[:, rows].cpu().double(), want.to(torch.bfloat16).double())
    assert torch.count_nonzero(y[-1]) == len(rows) and torch.count_nonzero(y[0]) == len(rows)


@pytest.mark.parametrize("m", [3, 40, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_subnormal_outputs(m, dtype):
    """Products below 2^-126: exact in float32, rounded to nearest in bfloat16."""
    import fp4_block_scaled_tensor_amd as fp4
    codes, scales = (v.reshape(-1) for v in np.meshgrid(np.arange(16), np.arange(0, 9)))
    w64 = OF.E2M1_VALUES[codes] * 2.0 ** (scales.astype(np.float64) - 127)
    x = rows_of([1.0, -1.5, 0.25, 1.9921875, 2.0 ** -8], m)              # 8 significant bits: exact in bf16
    want = x[:, 17].astype(np.float64)[:, None] * w64[None]
    w = one_product_weight(codes, scales)
    xd = torch.from_numpy(x).to(dtype).cuda()
    y = fp4.linear(xd, w, out_dtype=torch.float32).cpu().double().numpy()
    assert np.array_equal(y, want)                                          # multiples of 2^-149 all
    y = fp4.linear(xd, w, out_dtype=torch.bfloat16).cpu().double()
    assert torch.equal(y, torch.from_numpy(want).to(torch.float32).to(torch.bfloat16).double())
