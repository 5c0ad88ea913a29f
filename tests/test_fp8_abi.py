"""The 8-bit entry points on the host: header and binding agree, invalid arguments return their status before
anything is enqueued, and the binding's own checks (no GPU needed)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import fp4_block_scaled_tensor_amd as fp4
from fp4_block_scaled_tensor_amd import _lib, fp8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp4bs_fp8.h")
P, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4098)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libfp4bs.so is not built; run `python -m fp4_block_scaled_tensor_amd.build`")
    return _lib.load()


def test_header_and_binding_agree(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER, encoding="utf-8").read(), flags=re.S)
    decl = re.findall(r"^\s*fp4_status\s+(\w+)\s*\(", text, flags=re.M)
    assert sorted(decl) == sorted(_lib.FP8_EXPORTED) == sorted(_lib.FP8_SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True, text=True).stdout
    assert set(decl) <= {line.split()[-1] for line in out.splitlines() if " T " in line}


def test_quantize_rejects_bad_arguments(lib):
    def q(x=P, dt=0, rows=4, cols=200, ld=200, view=3, scale=0, q=P, s=P, qt=P, st=P):
        return lib.fp8_quantize(x, dt, rows, cols, ld, view, scale, q, s, qt, st, None)
    assert q(dt=2) == _lib.FP4_EINVAL
    assert q(scale=2) == _lib.FP4_EINVAL
    assert q(view=4) == _lib.FP4_EINVAL and q(view=-1) == _lib.FP4_EINVAL
    assert q(rows=-1) == _lib.FP4_EINVAL
    assert q(rows=1 << 31) == _lib.FP4_EUNSUPPORTED
    assert q(rows=1 << 20, cols=1 << 18, ld=1 << 18) == _lib.FP4_EUNSUPPORTED   # 2^24 tiles
    assert q(ld=199) == _lib.FP4_EINVAL
    assert q(ld=(1 << 22) + 1) == _lib.FP4_EUNSUPPORTED
    assert q(x=None) == _lib.FP4_EINVAL
    assert q(x=ctypes.c_void_p(4097)) == _lib.FP4_EALIGN
    assert q(x=ODD, dt=1) == _lib.FP4_EALIGN
    assert q(q=None) == _lib.FP4_EINVAL and q(s=None) == _lib.FP4_EINVAL
    assert q(qt=None) == _lib.FP4_EINVAL and q(st=None) == _lib.FP4_EINVAL
    assert q(view=2, qt=None) == _lib.FP4_EINVAL
    assert q(q=ctypes.c_void_p(4104)) == _lib.FP4_EALIGN
    assert q(scale=1, st=ODD) == _lib.FP4_EALIGN
    assert q(rows=0, x=None, q=None, s=None, qt=None, st=None) == _lib.FP4_OK


def op(q=P, s=P, scale=0, layout=0, rows=64, k=256):
    return ctypes.byref(_lib.F8Operand(q, s, scale, layout, rows, k))


def test_gemm_rejects_bad_arguments(lib):
    def g(a=None, b=None, y=P, dt=0, ld=64, ws=None, nb=0):
        return lib.fp8_gemm(a or op(rows=300), b or op(layout=1), y, dt, ld, ws, nb, None)
    assert lib.fp8_gemm(None, op(), P, 0, 64, None, 0, None) == _lib.FP4_EINVAL
    assert g(dt=2) == _lib.FP4_EINVAL
    assert g(a=op(layout=1)) == _lib.FP4_EUNSUPPORTED                   # the first operand needs 1D scales
    assert g(b=op(k=128)) == _lib.FP4_EINVAL
    assert g(b=op(scale=1)) == _lib.FP4_EUNSUPPORTED
    assert g(a=op(scale=2)) == _lib.FP4_EINVAL and g(b=op(layout=3)) == _lib.FP4_EINVAL
    assert g(a=op(rows=-1)) == _lib.FP4_EINVAL and g(a=op(k=-1)) == _lib.FP4_EINVAL
    assert g(a=op(rows=1 << 31)) == _lib.FP4_EUNSUPPORTED
    big = (1 << 22) + 128
    assert g(a=op(k=big), b=op(k=big)) == _lib.FP4_EUNSUPPORTED
    assert g(b=op(rows=1 << 30, k=256), ld=1 << 30) == _lib.FP4_EUNSUPPORTED   # its scales pass 32-bit offsets
    assert g(a=op(q=None)) == _lib.FP4_EINVAL and g(b=op(s=None)) == _lib.FP4_EINVAL
    assert g(a=op(q=ctypes.c_void_p(4104))) == _lib.FP4_EALIGN
    assert g(a=op(scale=1, s=ODD), b=op(scale=1)) == _lib.FP4_EALIGN
    assert g(ld=63) == _lib.FP4_EINVAL
    assert g(y=None) == _lib.FP4_EINVAL
    assert g(y=ODD, dt=1) == _lib.FP4_EALIGN
    nb = ctypes.c_size_t()
    w = lambda: op(layout=1, rows=4096, k=8192)   # noqa: E731
    assert lib.fp8_gemm_workspace(40, w(), 0, 0, 0, ctypes.byref(nb)) == _lib.FP4_OK and nb.value > 0
    assert g(a=op(rows=40, k=8192), b=w(), ld=4096, ws=P, nb=nb.value - 1) == _lib.FP4_EINVAL
    assert "workspace" in lib.fp4_last_error().decode()
    assert g(a=op(rows=40, k=8192), b=w(), ld=4096, ws=ctypes.c_void_p(4100), nb=nb.value) == _lib.FP4_EINVAL
    assert lib.fp8_gemm_workspace(40, None, 0, 0, 0, ctypes.byref(nb)) == _lib.FP4_EINVAL
    assert lib.fp8_gemm_workspace(40, w(), 0, 0, 0, None) == _lib.FP4_EINVAL
    assert lib.fp8_gemm_workspace(40, w(), 0, 3, 0, ctypes.byref(nb)) == _lib.FP4_EINVAL
    assert lib.fp8_gemm_workspace(40, w(), 1025, 0, 0, ctypes.byref(nb)) == _lib.FP4_EUNSUPPORTED
    assert g(a=op(rows=0)) == _lib.FP4_OK


def test_expert_gemm_rejects_bad_arguments(lib):
    def g(n=4, off=P, x=None, y=P):
        return lib.fp8_expert_gemm(x or op(rows=4), op(layout=1), n, off, y, 0, 64, None, 0, None)
    assert g(n=0) == _lib.FP4_EINVAL and g(n=1025) == _lib.FP4_EUNSUPPORTED
    assert g(off=None) == _lib.FP4_EINVAL and g(off=ODD) == _lib.FP4_EINVAL
    assert g(x=op(rows=0)) == _lib.FP4_OK


def test_gated_rejects_bad_arguments(lib):
    def g(n=0, off=None, act=0, h=P, kind=0, ld=32, hs=P, gu=None, gdt=0, ldgu=64, w=None):
        return lib.fp8_gated(op(rows=300), w or op(layout=1), n, off, act, h, kind, ld, hs, gu, gdt, ldgu, None, 0, None)
    assert g(act=3) == _lib.FP4_EINVAL and g(kind=3) == _lib.FP4_EINVAL
    assert g(w=op(layout=1, rows=63)) == _lib.FP4_EINVAL
    assert g(ld=31) == _lib.FP4_EINVAL
    assert g(kind=2, hs=None) == _lib.FP4_EINVAL and g(kind=2, h=ctypes.c_void_p(4104)) == _lib.FP4_EALIGN
    assert g(gu=P, gdt=2) == _lib.FP4_EINVAL and g(gu=P, ldgu=63) == _lib.FP4_EINVAL
    assert g(gu=ctypes.c_void_p(4097)) == _lib.FP4_EALIGN
    assert g(n=4) == _lib.FP4_EINVAL                                    # experts without offsets


def test_gated_grad_rejects_bad_arguments(lib):
    def plain(dh=P, dt=0, rows=4, f=100, lddh=100, gu=P, ldgu=200, act=0, dgu=P, ld=200):
        return lib.gated_grad(dh, dt, rows, f, lddh, gu, ldgu, act, dgu, ld, None)
    assert plain(dt=2) == _lib.FP4_EINVAL and plain(act=-1) == _lib.FP4_EINVAL
    assert plain(rows=-1) == _lib.FP4_EINVAL and plain(f=1 << 30, lddh=1 << 30) == _lib.FP4_EUNSUPPORTED
    assert plain(lddh=99) == _lib.FP4_EINVAL and plain(ldgu=199) == _lib.FP4_EINVAL and plain(ld=199) == _lib.FP4_EINVAL
    assert plain(dh=None) == _lib.FP4_EINVAL and plain(gu=None) == _lib.FP4_EINVAL and plain(dgu=None) == _lib.FP4_EINVAL
    assert plain(rows=0, dh=None, gu=None, dgu=None) == _lib.FP4_OK

    def views(f=128, scale=0, q=P, s=P, qt=P, st=P, rows=4):
        return lib.fp8_gated_grad(P, 0, rows, f, f, P, 2 * f, 0, scale, q, s, qt, st, None)
    assert views(f=100) == _lib.FP4_EUNSUPPORTED
    assert views(scale=2) == _lib.FP4_EINVAL
    assert views(q=None, qt=None) == _lib.FP4_EINVAL
    assert views(s=None) == _lib.FP4_EINVAL and views(st=None) == _lib.FP4_EINVAL
    assert views(qt=ctypes.c_void_p(4104)) == _lib.FP4_EALIGN
    assert views(rows=1 << 30, f=1 << 10) == _lib.FP4_EUNSUPPORTED


def test_binding_refuses(lib):
    x = torch.zeros(4, 128)
    with pytest.raises(ValueError, match="device tensors"):
        fp4.fp8_quantize(x)
    t = fp4.F8Tensor(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 1), fp4.FP4_SCALES_1D, 4, 128)
    for call in (lambda: fp4.fp8_gemm(t, t), lambda: fp4.fp8_gated(t, t), lambda: fp4.fp8_dequantize(t)):
        with pytest.raises(ValueError, match="device tensors"):
            call()
    with pytest.raises(ValueError):
        fp4.fp8_stack([])
    u = fp4.F8Tensor(t.q, t.s, fp4.FP4_SCALES_1D, 4, 100)
    with pytest.raises(ValueError, match="agree"):
        fp4.fp8_stack([t, u])
    with pytest.raises(ValueError, match="act"):
        fp8._act("relu")


def test_operand_checks():
    dev = torch.device("cpu")
    q = torch.zeros(4, 256, dtype=torch.uint8)
    good = lambda q=q, s=torch.zeros(4, 2), layout=0, rows=4, k=200: fp4.F8Tensor(q, s, layout, rows, k)   # noqa: E731
    assert fp8._operand(good(), "a", dev).scale == _lib.FP8_SCALE_F32
    assert fp8._operand(good(s=torch.zeros(4, 2, dtype=torch.uint8)), "a", dev).scale == _lib.FP8_SCALE_E8M0
    assert fp8._operand(good(s=torch.zeros(1, 2), layout=1), "a", dev).layout == 1
    for bad in (good(q=q[:, :128]), good(q=q.to(torch.int16)), good(q=q.t()), good(s=torch.zeros(4, 1)),
                good(s=torch.zeros(4, 2, dtype=torch.float16)), good(s=torch.zeros(2, 4).t()), good(rows=5), good(k=300)):
        with pytest.raises(ValueError):
            fp8._operand(bad, "a", dev)
    with pytest.raises(ValueError, match="on cuda"):
        fp8._operand(good(), "a", torch.device("cuda:0"))
    e = fp4.F8Experts(torch.zeros(3, 4, 256, dtype=torch.uint8), torch.zeros(3, 4, 2), 0, 4, 200)
    assert e.n_experts == 3 and fp8._operand(e, "w", dev, 3).rows == 4
    with pytest.raises(ValueError):
        fp8._operand(fp4.F8Experts(e.q, e.s[:2], 0, 4, 200), "w", dev, 3)
