"""Edges of the mixture-of-experts operators: no tokens with any number of experts."""
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
