"""Edges of the mixture-of-experts operators: no tokens with any number of experts, every bit pattern of a
gathered row."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("experts", [1, 5, 511, 512, 513, 1000, 1024])
@pytest.mark.parametrize("ids64", [0, 1])
def test_sort_without_tokens_writes_the_offsets(experts, ids64):
    """tokens = 0: every offset is zero, nothing past them is written, through the C entry without a workspace."""
    from fp4_block_scaled_tensor_amd import _lib
    import fp4_block_scaled_tensor_amd as fp4
    offsets = torch.full((experts + 9,), -7, dtype=torch.int32, device="cuda")
    _lib.check(fp4.library().fp4_expert_sort(None, ids64, 0, 2, 2, experts, None, None, offsets.data_ptr(), None, 0,
                                             None))
    torch.cuda.synchronize()
    assert offsets.cpu().tolist() == [0] * (experts + 1) + [-7] * 8
    plan = fp4.expert_sort(torch.empty((0, 2), dtype=torch.int32, device="cuda"), experts)
    assert plan.offsets.cpu().tolist() == [0] * (experts + 1) and plan.pos.shape == (0, 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hidden,pad", [(4096, 0), (4093, 3), (7, 0)])
def test_gather_copies_bits(hidden, pad, dtype):
    """A gathered row is its token's row bit for bit: subnormals, signed zeros, and NaNs with their payloads."""
    import fp4_block_scaled_tensor_amd as fp4
    r = np.random.Generator(np.random.PCG64(hidden))
    tokens, topk, experts = 33, 3, 4
    if dtype == "bf16":
        bits = (np.arange(tokens * hidden, dtype=np.int64) * 40503 % 65536).astype(np.uint16).view(np.int16).reshape(tokens, hidden)
        kind = torch.bfloat16
    else:
        bits = r.integers(0, 2 ** 32, (tokens, hidden), dtype=np.uint32)
        nan = r.random((tokens, hidden)) < 0.2
        bits = np.where(nan, bits | np.uint32(0x7F800000), bits).astype(np.uint32).view(np.int32)
        kind = torch.float32
    x = torch.zeros((tokens, hidden + pad), dtype=torch.from_numpy(bits).dtype, device="cuda")
    x[:, :hidden] = torch.from_numpy(bits).cuda()
    ids = torch.from_numpy(r.integers(-1, experts, (tokens, topk)).astype(np.int32)).cuda()
    plan = fp4.expert_sort(ids, experts)
    xs = fp4.expert_gather(x.view(kind)[:, :hidden], plan)
    order, kept = plan.order.cpu().numpy(), int(plan.offsets[-1])
    want = np.zeros((tokens * topk, hidden), bits.dtype)
    want[:kept] = bits[order[:kept] // topk]
    assert np.array_equal(xs.view(x.dtype).cpu().numpy(), want)


def test_sort_of_almost_2_to_the_31_slots():
    """The largest number of slots: the last wave's range ends at 2^31 - 1. All slots of expert 0 but the first, the
    middle one and the last (expert 1), so every position is known."""
    import fp4_block_scaled_tensor_amd as fp4
    n = 2 ** 31 - 1
    mid = n // 2
    ids = torch.zeros((n, 1), dtype=torch.int32, device="cuda")
    for s in (0, mid, n - 1):
        ids[s] = 1
    plan = fp4.expert_sort(ids, 2)
    assert plan.offsets.cpu().tolist() == [0, n - 3, n]
    order, pos = plan.order, plan.pos.view(-1)
    assert order[-3:].cpu().tolist() == [0, mid, n - 1]
    assert pos[0] == n - 3 and pos[mid] == n - 2 and pos[n - 1] == n - 1
    step = 2 ** 27
    for lo in range(0, n - 3, step):                      # position p holds slot p + 1, from the middle on p + 2
        hi = min(lo + step, n - 3)
        p = torch.arange(lo, hi, device="cuda")
        slot = p + 1 + (p + 1 >= mid)
        assert torch.equal(order[lo:hi].long(), slot), lo
        assert torch.equal(pos[slot].long(), p), lo


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sums_keep_subnormals(dtype):
    """Subnormal rows come through the sums and the gradients: with one slot to a token and weights of 1 every output
    is its input; two equal slots double it (exactly, also where the result is subnormal)."""
    import fp4_block_scaled_tensor_amd as fp4
    kind, word, count = (torch.bfloat16, torch.int16, 127) if dtype == "bf16" else (torch.float32, torch.int32, 2 ** 23 - 1)
    bits = torch.arange(1, count + 1, max(1, count // 4000), dtype=torch.int64)
    bits = torch.cat([bits, bits + (2 ** 15 if dtype == "bf16" else 2 ** 31)])                    # both signs
    bits = torch.where(bits >= 2 ** (8 * word.itemsize - 1), bits - 2 ** (8 * word.itemsize), bits).to(word)
    rows = bits.view(kind).repeat(2, 1).cuda()
    one = fp4.expert_sort(torch.tensor([[1], [0]], dtype=torch.int32, device="cuda"), 2)
    w = torch.ones((2, 1), device="cuda")
    flip = rows.flip(0)
    same = lambda a, b: torch.equal(a.contiguous().view(word), b.contiguous().view(word))   # noqa: E731
    assert same(fp4.expert_gather_grad(rows, one), flip) and same(fp4.expert_combine(rows, w, one), flip)
    dys, _ = fp4.expert_combine_grad(rows, rows, w, one)
    assert same(dys, flip)
    two = fp4.expert_sort(torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), 2)
    twice = (rows[:1].double() * 2).to(kind)
    assert same(fp4.expert_gather_grad(rows, two), twice)
    assert same(fp4.expert_combine(rows, torch.ones((1, 2), device="cuda"), two), twice)
