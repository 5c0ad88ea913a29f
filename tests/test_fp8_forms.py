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
