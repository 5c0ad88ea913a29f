"""The mixture-of-experts entry points on the host: the header and the binding agree, and invalid
arguments return their status before anything is enqueued (no GPU needed)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from fp4_block_scaled_tensor_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp4bs_experts.h")
P = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libfp4bs.so is not built; run `python -m fp4_block_scaled_tensor_amd.build`")
    return _lib.load()


def test_header_and_binding_agree(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER, encoding="utf-8").read(), flags=re.S)
    decl = re.findall(r"^\s*fp4_status\s+(\w+)\s*\(", text, flags=re.M)
    assert sorted(decl) == sorted(_lib.EXPERTS_EXPORTED) == sorted(_lib.EXPERTS_SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True, text=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert set(decl) <= exported


def test_sort_rejects_bad_arguments(lib):
    def sort(ids=P, i64=0, tokens=4, topk=2, ld=2, experts=8, order=P, pos=P, offsets=P, ws=None, nb=0):
        return lib.fp4_expert_sort(ids, i64, tokens, topk, ld, experts, order, pos, offsets, ws, nb, None)
    assert sort(i64=2) == _lib.FP4_EINVAL
    assert sort(tokens=-1) == _lib.FP4_EINVAL
    assert sort(topk=0) == _lib.FP4_EINVAL
    assert sort(tokens=1 << 30, topk=2) == _lib.FP4_EUNSUPPORTED       # 2^31 slots
    assert sort(experts=0) == _lib.FP4_EINVAL
    assert sort(experts=1025) == _lib.FP4_EUNSUPPORTED
    assert sort(ld=1) == _lib.FP4_EINVAL                               # row stride < topk
    assert sort(ids=None) == _lib.FP4_EINVAL
    assert sort(ids=ctypes.c_void_p(4100), i64=1) == _lib.FP4_EALIGN
    assert sort(order=None) == _lib.FP4_EINVAL
    assert sort(pos=ctypes.c_void_p(4098)) == _lib.FP4_EINVAL
    assert sort(offsets=None) == _lib.FP4_EINVAL
    assert sort(tokens=100000) == _lib.FP4_EINVAL                      # needs a workspace
    assert "workspace" in lib.fp4_last_error().decode()
    nb = ctypes.c_size_t()
    assert lib.fp4_expert_sort_workspace(100000, 2, 8, ctypes.byref(nb)) == _lib.FP4_OK and nb.value > 0
    assert sort(tokens=100000, ws=P, nb=nb.value - 1) == _lib.FP4_EINVAL
    assert lib.fp4_expert_sort_workspace(4, 2, 8, None) == _lib.FP4_EINVAL
    assert lib.fp4_expert_sort_workspace(4, 2, 0, ctypes.byref(nb)) == _lib.FP4_EINVAL


def test_row_moves_reject_bad_arguments(lib):
    def gather(x=P, dt=0, tokens=4, hidden=64, ldx=64, pos=P, topk=2, xs=P, ldxs=64, name="fp4_expert_gather"):
        return getattr(lib, name)(x, dt, tokens, hidden, ldx, pos, topk, xs, ldxs, None)
    for name in ("fp4_expert_gather", "fp4_expert_gather_grad"):
        assert gather(dt=5, name=name) == _lib.FP4_EINVAL
        assert gather(tokens=-1, name=name) == _lib.FP4_EINVAL
        assert gather(hidden=-1, name=name) == _lib.FP4_EINVAL
        assert gather(topk=0, name=name) == _lib.FP4_EINVAL
        assert gather(tokens=1 << 30, name=name) == _lib.FP4_EUNSUPPORTED
        assert gather(ldx=63, name=name) == _lib.FP4_EINVAL
        assert gather(ldxs=63, name=name) == _lib.FP4_EINVAL
        assert gather(x=None, name=name) == _lib.FP4_EINVAL
        assert gather(xs=None, name=name) == _lib.FP4_EINVAL
        assert gather(x=ctypes.c_void_p(4097), name=name) == _lib.FP4_EALIGN
        assert gather(dt=1, xs=ctypes.c_void_p(4098), name=name) == _lib.FP4_EALIGN
        assert gather(pos=None, name=name) == _lib.FP4_EINVAL
        assert gather(x=None, xs=None, pos=None, tokens=0, name=name) == _lib.FP4_OK      # empty: no-op

    def combine(w=P, ldw=2, ys=P, y=P):
        return lib.fp4_expert_combine(ys, 0, 4, 64, 64, w, ldw, P, 2, y, 64, None)
    assert combine(w=None) == _lib.FP4_EINVAL
    assert combine(w=ctypes.c_void_p(4098)) == _lib.FP4_EALIGN
    assert combine(ldw=1) == _lib.FP4_EINVAL
    assert combine(y=None) == _lib.FP4_EINVAL

    def grad(dy=P, ys=P, w=P, dys=P, dw=P, lddw=2, dt=0, pos=P):
        return lib.fp4_expert_combine_grad(dy, dt, 4, 64, 64, ys, 64, w, 2, pos, 2, dys, 64, dw, lddw, None)
    assert grad(dt=9) == _lib.FP4_EINVAL
    assert grad(dy=None) == _lib.FP4_EINVAL
    assert grad(ys=None) == _lib.FP4_EINVAL                            # dw needs ys
    assert grad(w=None) == _lib.FP4_EINVAL                             # dys needs w
    assert grad(lddw=1) == _lib.FP4_EINVAL
    assert grad(dw=ctypes.c_void_p(4098)) == _lib.FP4_EALIGN
    assert grad(pos=ctypes.c_void_p(4098)) == _lib.FP4_EINVAL
    assert grad(dys=None, dw=None) == _lib.FP4_OK                      # nothing asked for


def op(rows=64, k=128, fmt=0, block=16, layout=0, q=4096, s=4096, g=None, stripe=0):
    return _lib.Operand(q, s, g, fmt, block, layout, stripe, rows, k)


def test_linear_rejects_bad_arguments(lib):
    def linear(x=P, xdt=0, rows=4, ldx=128, w=None, y=P, ydt=0, ldy=64, experts=None, offsets=P):
        w = op() if w is None else w
        if experts is None:
            return lib.fp4_linear(x, xdt, rows, ldx, ctypes.byref(w), y, ydt, ldy, None, 0, None)
        return lib.fp4_expert_linear(x, xdt, rows, ldx, ctypes.byref(w), experts, offsets, y, ydt, ldy, None, 0, None)
    for experts in (None, 8):
        assert linear(xdt=3, experts=experts) == _lib.FP4_EINVAL
        assert linear(ydt=3, experts=experts) == _lib.FP4_EINVAL
        assert linear(rows=-1, experts=experts) == _lib.FP4_EINVAL
        assert linear(rows=1 << 31, experts=experts) == _lib.FP4_EUNSUPPORTED
        assert linear(ldx=127, experts=experts) == _lib.FP4_EINVAL
        assert linear(ldx=129, experts=experts) == _lib.FP4_EALIGN             # rows of x not 16-byte aligned
        assert linear(x=ctypes.c_void_p(4104), experts=experts) == _lib.FP4_EALIGN
        assert linear(x=None, experts=experts) == _lib.FP4_EINVAL
        assert linear(y=None, experts=experts) == _lib.FP4_EINVAL
        assert linear(ldy=63, experts=experts) == _lib.FP4_EINVAL
        assert linear(ydt=1, y=ctypes.c_void_p(4098), experts=experts) == _lib.FP4_EALIGN
        assert linear(w=op(k=96), ldx=96, experts=experts) == _lib.FP4_EINVAL   # K % 64
        assert linear(w=op(fmt=2), experts=experts) == _lib.FP4_EUNSUPPORTED    # E8M0 with block 16
        assert linear(w=op(fmt=7), experts=experts) == _lib.FP4_EINVAL
        assert linear(w=op(q=4100), experts=experts) == _lib.FP4_EALIGN
        assert linear(w=op(s=4098), experts=experts) == _lib.FP4_EALIGN         # scales read as words
        assert linear(w=op(layout=1, rows=40), ldy=40, experts=experts) == _lib.FP4_EINVAL   # 2D rows % 16
        assert linear(w=op(stripe=16), experts=experts) == _lib.FP4_EINVAL      # stripes without g
        assert linear(rows=0, x=None, y=None, experts=experts) == _lib.FP4_OK   # empty: no-op
    assert linear(experts=0) == _lib.FP4_EINVAL
    assert linear(experts=1025) == _lib.FP4_EUNSUPPORTED
    assert linear(experts=8, offsets=None) == _lib.FP4_EINVAL
    assert lib.fp4_linear(P, 0, 4, 128, None, P, 0, 64, None, 0, None) == _lib.FP4_EINVAL
    nb = ctypes.c_size_t()
    assert lib.fp4_linear_workspace(4, 0, ctypes.byref(op()), 0, None) == _lib.FP4_EINVAL
    assert lib.fp4_linear_workspace(4, 9, ctypes.byref(op()), 0, ctypes.byref(nb)) == _lib.FP4_EINVAL
    assert lib.fp4_linear_workspace(4, 0, ctypes.byref(op()), 1025, ctypes.byref(nb)) == _lib.FP4_EUNSUPPORTED
    assert lib.fp4_linear_workspace(4, 0, ctypes.byref(op()), 0, ctypes.byref(nb)) == _lib.FP4_OK


def test_binding_rejects_host_tensors_and_bad_shapes():
    import fp4_block_scaled_tensor_amd as fp4
    ids = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensors"):
        fp4.expert_sort(ids, 8)
    plan = fp4.ExpertPlan(ids.view(-1), ids, torch.zeros(9, dtype=torch.int32), 4, 2, 8)
    with pytest.raises(ValueError, match="device tensors"):
        fp4.expert_gather(torch.zeros(4, 64), plan)
    with pytest.raises(ValueError, match="device tensors"):
        fp4.expert_combine(torch.zeros(8, 64), torch.zeros(4, 2), plan)
    w = fp4.QTensor(torch.zeros((32, 32), dtype=torch.uint8), torch.zeros((32, 4), dtype=torch.uint8), torch.ones(1),
                    fp4.UE5M3, 16, fp4.FP4_SCALES_1D, 32, 64)
    with pytest.raises(ValueError, match="device tensors"):
        fp4.linear(torch.zeros(4, 64), w)
    with pytest.raises(ValueError, match="no weights"):
        fp4.stack_experts([])
    v = fp4.QTensor(w.q, w.s, w.g, fp4.E4M3, 16, fp4.FP4_SCALES_1D, 32, 64)
    with pytest.raises(ValueError, match="must agree"):
        fp4.stack_experts([w, v])
    stack = fp4.stack_experts([w, w, w])
    assert stack.n_experts == 3 and stack.q.shape == (3, 32, 32) and stack.g.shape == (3, 1)
