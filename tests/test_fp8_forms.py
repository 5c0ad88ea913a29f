"""The forms of the 8-bit products on the host: the sizes that the GPU tests compare take every one that calls reach,
by the same choice that the calls make (no GPU needed: a device of 256 compute units is assumed without one)."""
import ctypes
import itertools

import pytest

from fp4_block_scaled_tensor_amd import _lib
from tests import _fp8_forms as F

ROWS = (1, 3, 9, 17, 33, 64, 100, 129, 200, 400, 515, 900, 1500, 2047, 4100, 6144, 8192)
WEIGHT = (64, 200, 520, 1030, 2048, 4096, 6144, 14336, 28672)
K = (128, 300, 1100, 2048, 4096, 8191, 14336, 32768)


@pytest.mark.parametrize("experts", [(0,), (2, 8, 32)])
@pytest.mark.parametrize("gated", [False, True])
def test_every_form_is_compared(gated, experts):
    compared = set().union(*(F.forms(s, gated) for s in (F.GATED if gated else F.GEMM)))
    for m, n, k, e in itertools.product(ROWS, WEIGHT, K, experts):
        missing = F.forms((m, n, k, e), gated) - compared
        assert not missing, ((m, n, k, e), missing)


def test_form_and_workspace_agree():
    """Sums of a split K and turned scales are what the workspace holds."""
    lib, nb = _lib.load(), ctypes.c_size_t()
    for m, n, k, e in F.GEMM:
        w = _lib.F8Operand(None, None, _lib.FP8_SCALE_E8M0, _lib.FP4_SCALES_2D, n, k)
        _lib.check(lib.fp8_gemm_workspace(m, ctypes.byref(w), e, 0, 0, ctypes.byref(nb)))
        _, _, parts, turned = F.form(m, n, k, e, 0, 0)
        scales = -(-m * -(-k // 128) // 256) * 256 if turned else 0
        assert nb.value == scales + (parts * m * n * 4 if parts > 1 else 0), (m, n, k, e)


def test_form_refuses():
    lib, f = _lib.load(), (ctypes.c_int32 * 4)()
    w = lambda **kw: ctypes.byref(_lib.F8Operand(None, None, **dict(dict(scale=0, layout=1, rows=64, k=256), **kw)))   # noqa: E731
    assert lib.fp8_gemm_form(4, None, 0, 0, 0, f) == _lib.FP4_EINVAL
    assert lib.fp8_gemm_form(4, w(), 0, 3, 0, f) == _lib.FP4_EINVAL and lib.fp8_gemm_form(4, w(), 0, 0, 2, f) == _lib.FP4_EINVAL
    assert lib.fp8_gemm_form(4, w(), 0, 0, 0, None) == _lib.FP4_EINVAL
    assert lib.fp8_gemm_form(4, w(scale=2), 0, 0, 0, f) == _lib.FP4_EINVAL
    assert lib.fp8_gemm_form(4, w(rows=63), 0, 1, 0, f) == _lib.FP4_EINVAL
    assert lib.fp8_gemm_form(4, w(), 1025, 0, 0, f) == _lib.FP4_EUNSUPPORTED
    assert lib.fp8_gemm_form(0, w(), 0, 0, 0, f) == _lib.FP4_OK and tuple(f) == (0, 0, 0, 0)


def status(m, n, k, experts=0, gated=0, f32=0):
    f = (ctypes.c_int32 * 4)()
    w = _lib.F8Operand(None, None, _lib.FP8_SCALE_E8M0, _lib.FP4_SCALES_2D, n, k)
    st = _lib.load().fp8_gemm_form(m, ctypes.byref(w), experts, gated, f32, f)
    return st, tuple(f)


@pytest.mark.parametrize("f32", [0, 1])
@pytest.mark.parametrize("n,k", [(64, 128), (200, 128), (256, 256), (4096, 512), (100000, 128)])
def test_the_largest_launches(n, k, f32):
    """What is accepted has fewer than 2^32 threads, by the tiles that the call says it takes; what is refused is past
    the tiles that are always accepted, and says why."""
    div = lambda a, b: -(-a // b)   # noqa: E731
    for log in range(20, 31):
        for m in (1 << log, (1 << log) + (1 << log - 1), (1 << log + 1) - 1):
            st, (bm, bn, parts, _) = status(m, n, k, f32=f32)
            if st == _lib.FP4_OK:
                assert div(m, bm) * div(n, bn) * parts * (512 if bm >= 128 else 256) < 1 << 32, m
            else:
                assert st == _lib.FP4_EUNSUPPORTED and "tiles" in _lib.load().fp4_last_error().decode()
                assert div(m, 32) * div(n, 128) >= 1 << 22, m
    for e in (1, 1024):
        assert status(1 << 20, 256, k, experts=e, f32=f32)[0] == _lib.FP4_OK
