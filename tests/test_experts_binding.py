"""What the binding of the mixture-of-experts operators hands to the library, seen by a library that
only records (no GPU needed): the tensors behind the pointers it gets."""
import ctypes
import gc

import pytest
import torch

from fp4_block_scaled_tensor_amd import _lib, experts
import fp4_block_scaled_tensor_amd as fp4


class Recorder:
    """The built library for workspace sizes; every other entry point runs `seen(name, args)` and succeeds."""

    def __init__(self, seen):
        self.lib, self.seen = _lib.load(), seen

    def __getattr__(self, name):
        if name.endswith("_workspace"):
            return getattr(self.lib, name)

        def call(*args):
            self.seen(name, args)
            return _lib.FP4_OK
        return call


@pytest.fixture
def record(monkeypatch):
    """Host tensors stand for device tensors."""
    def start(seen):
        rec = Recorder(seen)
        monkeypatch.setattr(_lib, "load", lambda: rec)
        monkeypatch.setattr(experts, "_dev_check", lambda *a: None)
        monkeypatch.setattr(experts, "_stream_of", lambda *a: 0)
    return start


def owners(address):
    """Live tensors that own the memory at address."""
    return [t for t in gc.get_objects() if isinstance(t, torch.Tensor) and t.numel() and t.data_ptr() == address]


def weight(n, k, count=None):
    """An MXFP4 weight of zeros, or a stack of them."""
    if count is None:
        return fp4.QTensor(torch.zeros((n, k // 2), dtype=torch.uint8), torch.full((n, k // 32), 127, dtype=torch.uint8),
                           torch.ones(1), fp4.E8M0, 32, fp4.FP4_SCALES_1D, n, k)
    return fp4.stack_experts([weight(n, k) for _ in range(count)])


# (call, position of the workspace among the library call's arguments)
WITH_WORKSPACE = {
    "sort": (lambda: fp4.expert_sort(torch.zeros((9000, 2), dtype=torch.int32), 8), 9),
    "linear_f32": (lambda: fp4.linear(torch.zeros(3, 128), weight(32, 128)), 8),
    "linear_split": (lambda: fp4.linear(torch.zeros((40, 4096), dtype=torch.bfloat16), weight(64, 4096)), 8),
    "experts_f32": (lambda: fp4.expert_linear(torch.zeros(60, 1024), weight(32, 1024, 2),
                                              torch.tensor([0, 20, 60], dtype=torch.int32)), 10),
}


@pytest.mark.parametrize("case", WITH_WORKSPACE)
def test_workspace_lives_until_the_call_has_returned(case, record):
    """The allocator may hand a dropped workspace to another thread while the library is still enqueuing its kernels."""
    call, at = WITH_WORKSPACE[case]
    found = []

    def seen(name, args):
        found.append((name, args[at], args[at + 1], len(owners(args[at]))))
    record(seen)
    call()
    assert len(found) == 1
    name, ws, size, alive = found[0]
    assert ws and size > 0, f"{name} got no workspace: the case does not test anything"
    assert alive, f"{name}: the workspace tensor was gone before the call"


# ------------------------------------------------------------------ plans

def plan_of(tokens=4, topk=2, experts=3, **changes):
    n = tokens * topk
    made = dict(order=torch.arange(n, dtype=torch.int32), pos=torch.arange(n, dtype=torch.int32).view(tokens, topk),
                offsets=torch.tensor([0] + [n] * experts, dtype=torch.int32), tokens=tokens, topk=topk, n_experts=experts)
    return fp4.ExpertPlan(**(made | changes))


ROW_CALLS = {
    "gather": lambda plan: fp4.expert_gather(torch.zeros(4, 8), plan),
    "gather_grad": lambda plan: fp4.expert_gather_grad(torch.zeros(8, 8), plan),
    "combine": lambda plan: fp4.expert_combine(torch.zeros(8, 8), torch.zeros(4, 2), plan),
    "combine_grad": lambda plan: fp4.expert_combine_grad(torch.zeros(4, 8), torch.zeros(8, 8), torch.zeros(4, 2), plan),
}
BAD_POS = {
    "int64": torch.zeros((4, 2), dtype=torch.int64),
    "short": torch.zeros((3, 2), dtype=torch.int32),
    "long": torch.zeros((5, 2), dtype=torch.int32),
    "strided": torch.zeros((4, 5), dtype=torch.int32)[:, :2],
    "transposed": torch.zeros((2, 4), dtype=torch.int32).t(),
    "elsewhere": torch.zeros((4, 2), dtype=torch.int32, device="meta"),
}


@pytest.mark.parametrize("call", ROW_CALLS)
@pytest.mark.parametrize("bad", BAD_POS)
def test_row_moves_check_the_plans_positions(call, bad, record):
    """ExpertPlan is built by callers, too: the kernels read pos as packed int32 [tokens, topk] of x's device."""
    names = []
    record(lambda name, args: names.append(name))
    ROW_CALLS[call](plan_of())
    ROW_CALLS[call](plan_of(pos=torch.arange(8, dtype=torch.int32)))     # packed in slot order: the same memory
    assert names == [f"fp4_expert_{call}"] * 2
    with pytest.raises(ValueError, match="pos"):
        ROW_CALLS[call](plan_of(pos=BAD_POS[bad]))
    assert len(names) == 2, "enqueued in spite of the refusal"


@pytest.mark.parametrize("rows", [7, 9, 0])
def test_expert_linear_wants_the_plans_rows(rows, record):
    """With a plan x has its rows, tokens * topk; with offsets alone any number of them."""
    names = []
    record(lambda name, args: names.append(name))
    w = weight(32, 128, 3)
    x = torch.zeros((rows, 128), dtype=torch.bfloat16)
    fp4.expert_linear(torch.zeros((8, 128), dtype=torch.bfloat16), w, plan_of())
    fp4.expert_linear(x, w, plan_of().offsets)
    assert names == ["fp4_expert_linear"] * 2
    with pytest.raises(ValueError, match="8"):
        fp4.expert_linear(x, w, plan_of())
    assert len(names) == 2


@pytest.mark.parametrize("offsets", [torch.zeros(4, dtype=torch.int64), torch.zeros(3, dtype=torch.int32),
                                     torch.zeros(8, dtype=torch.int32)[::2],
                                     torch.zeros(4, dtype=torch.int32, device="meta")], ids=str)
def test_expert_linear_checks_the_offsets(offsets, record):
    names = []
    record(lambda name, args: names.append(name))
    with pytest.raises(ValueError, match="offsets"):
        fp4.expert_linear(torch.zeros((8, 128), dtype=torch.bfloat16), weight(32, 128, 3), offsets)
    assert not names
