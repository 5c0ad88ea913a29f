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


# ------------------------------------------------------------------ devices

class On:
    """Stands for a tensor of CUDA device `index`."""

    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index


def test_calls_run_with_their_tensors_device_current(monkeypatch):
    """The library launches on the current device, so the first tensor's is made current around the call."""
    now = [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *exc):
            now[0] = self.before
    monkeypatch.setattr(experts, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)

    @experts._on_its_device
    def call(x, factor=1):
        """doc"""
        if factor < 0:
            raise ValueError("refused")
        return now[0], x.index * factor
    assert call(On(0)) == (0, 0) and call(On(2)) == (2, 2) and call(x=On(3), factor=2) == (3, 6)
    with pytest.raises(ValueError, match="refused"):
        call(On(1), -1)
    assert now == [0] and call.__doc__ == "doc"
    assert call(On(-1)) == (0, -1)          # a host tensor: the call itself refuses it


@pytest.mark.parametrize("name", ["expert_sort", "expert_gather", "expert_gather_grad", "expert_combine",
                                  "expert_combine_grad", "linear", "expert_linear"])
def test_every_entry_point_makes_its_device_current(name):
    assert getattr(fp4, name).__wrapped__.__name__ == name


def on_meta(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype, device="meta")


ELSEWHERE = {
    "gather_out": lambda: fp4.expert_gather(torch.zeros(4, 8), plan_of(), out=on_meta(8, 8)),
    "gather_grad_out": lambda: fp4.expert_gather_grad(torch.zeros(8, 8), plan_of(), out=on_meta(4, 8)),
    "combine_weights": lambda: fp4.expert_combine(torch.zeros(8, 8), on_meta(4, 2), plan_of()),
    "combine_out": lambda: fp4.expert_combine(torch.zeros(8, 8), torch.zeros(4, 2), plan_of(), out=on_meta(4, 8)),
    "grad_ys": lambda: fp4.expert_combine_grad(torch.zeros(4, 8), on_meta(8, 8), torch.zeros(4, 2), plan_of()),
    "grad_weights": lambda: fp4.expert_combine_grad(torch.zeros(4, 8), torch.zeros(8, 8), on_meta(4, 2), plan_of()),
    "linear_out": lambda: fp4.linear(torch.zeros(4, 128), weight(32, 128), out=on_meta(4, 32)),
    "experts_out": lambda: fp4.expert_linear(torch.zeros(8, 128), weight(32, 128, 3), plan_of(), out=on_meta(8, 32)),
}


@pytest.mark.parametrize("case", ELSEWHERE)
def test_tensors_of_one_call_share_a_device(case, record):
    names = []
    record(lambda name, args: names.append(name))
    with pytest.raises(ValueError, match="must be on cpu"):
        ELSEWHERE[case]()
    assert not names


# ------------------------------------------------------------------ weights

def replaced(w, **changes):
    import dataclasses
    return dataclasses.replace(w, **changes)


BAD_WEIGHTS = {
    "payload_type": lambda w: replaced(w, q=w.q.to(torch.int32)),
    "payload_short": lambda w: replaced(w, q=w.q[..., :-1, :].contiguous()),
    "payload_strided": lambda w: replaced(w, q=torch.zeros((*w.q.shape[:-1], 2 * w.q.shape[-1]), dtype=torch.uint8)[..., ::2]),
    "payload_elsewhere": lambda w: replaced(w, q=w.q.to("meta")),
    "scales_type": lambda w: replaced(w, s=w.s.to(torch.int32)),
    "scales_short": lambda w: replaced(w, s=w.s[..., :-1].contiguous()),
    "scales_strided": lambda w: replaced(w, s=w.s.transpose(-1, -2)),
    "scales_elsewhere": lambda w: replaced(w, s=w.s.to("meta")),
    "g_type": lambda w: replaced(w, g=w.g.double()),
    "g_short": lambda w: replaced(w, g=w.g[..., :-1].contiguous()),
    "g_elsewhere": lambda w: replaced(w, g=w.g.to("meta")),
}


def ue5m3_weight(n, k, count=None, layout=None, stripe=32):
    layout = fp4.FP4_SCALES_1D if layout is None else layout
    if count is not None:
        return fp4.stack_experts([ue5m3_weight(n, k, None, layout, stripe) for _ in range(count)])
    shape = {fp4.FP4_SCALES_1D: (n, k // 16), fp4.FP4_SCALES_2D: (n // 16, k // 16),
             fp4.FP4_SCALES_2D_T: (k // 16, n // 16)}[layout]
    return fp4.QTensor(torch.zeros((n, k // 2), dtype=torch.uint8), torch.zeros(shape, dtype=torch.uint8),
                       torch.ones(-(-n // stripe) if stripe else 1), fp4.UE5M3, 16, layout, n, k, stripe)


@pytest.mark.parametrize("bad", BAD_WEIGHTS)
@pytest.mark.parametrize("count", [None, 3])
def test_products_check_the_weights_buffers(bad, count, record):
    """QTensor and ExpertWeights are built by callers, too: the kernels read their buffers as packed codes of the
    sizes that rows, k, block, layout and g_stripe say."""
    names = []
    record(lambda name, args: names.append(name))
    x = torch.zeros((8, 128), dtype=torch.bfloat16)

    def call(w):
        return fp4.linear(x, w) if count is None else fp4.expert_linear(x, w, plan_of())
    w = ue5m3_weight(80, 128, count)
    call(w)
    assert len(names) == 1
    with pytest.raises(ValueError, match="payload|scales|g "):
        call(BAD_WEIGHTS[bad](w))
    assert len(names) == 1


@pytest.mark.parametrize("count", [None, 3])
def test_every_form_of_a_weight_is_taken(count, record):
    names = []
    record(lambda name, args: names.append(name))
    x = torch.zeros((8, 128), dtype=torch.bfloat16)
    weights = [weight(37, 128, count), ue5m3_weight(37, 128, count, stripe=0), ue5m3_weight(37, 128, count, stripe=16),
               ue5m3_weight(48, 128, count, fp4.FP4_SCALES_2D, 0), ue5m3_weight(48, 128, count, fp4.FP4_SCALES_2D_T, 0),
               weight(0, 128, count)]
    weights.append(replaced(weights[1], g=weights[1].g[..., :0]))     # no tensor scale: 1
    for w in weights:
        fp4.linear(x, w) if count is None else fp4.expert_linear(x, w, plan_of())
    assert len(names) == len(weights)
    if count:
        with pytest.raises(ValueError, match="payload"):             # an expert's codes must follow each other
            fp4.expert_linear(x, replaced(weights[0], q=torch.zeros((3, 40, 64), dtype=torch.uint8)), plan_of())


# ------------------------------------------------------------------ sizes

def test_products_refuse_more_tiles_than_a_launch_holds():
    """A grid of 2^32 threads or more is cut off without an error, so the library refuses it from the sizes alone."""
    lib, nb = _lib.load(), ctypes.c_size_t()

    def workspace(rows, n, k, count, dtype=0):
        op = _lib.Operand(None, None, None, fp4.E8M0, 32, fp4.FP4_SCALES_1D, 0, n, k)
        return lib.fp4_linear_workspace(rows, dtype, ctypes.byref(op), count, ctypes.byref(nb))
    assert workspace(1, 2 ** 31 - 1, 64, 0) == _lib.FP4_OK
    assert workspace(20, 2 ** 31 - 1, 64, 0) == _lib.FP4_OK
    assert workspace(2 ** 20, 2 ** 17, 64, 0) == _lib.FP4_OK           # 2^21 tiles of 256 x 256
    assert workspace(1024, 2 ** 22, 64, 1024) == _lib.FP4_OK           # few rows: no tiles
    assert workspace(1, 2 ** 30, 64, 0) == _lib.FP4_OK
    assert workspace(17 * 1024, 2 ** 23, 64, 1024) == _lib.FP4_EUNSUPPORTED
    assert "one launch" in lib.fp4_last_error().decode()
    op = _lib.Operand(4096, 4096, None, fp4.E8M0, 32, fp4.FP4_SCALES_1D, 0, 2 ** 23, 64)
    p = ctypes.c_void_p(4096)
    assert lib.fp4_expert_linear(p, 0, 17 * 1024, 64, ctypes.byref(op), 1024, p, p, 0, 2 ** 23, p, 1 << 40,
                                 None) == _lib.FP4_EUNSUPPORTED
