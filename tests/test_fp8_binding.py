"""The 8-bit operators' binding on the host: operands by keyword, and what may be an operand (no GPU needed)."""
import ctypes

import pytest
import torch

import fp4_block_scaled_tensor_amd as fp4
from fp4_block_scaled_tensor_amd import _lib, fp8


def host_operand(rows=4, k=128):
    return fp4.F8Tensor(torch.zeros(rows, k, dtype=torch.uint8), torch.zeros(rows, 1), fp4.FP4_SCALES_1D, rows, k)


def host_stack():
    return fp4.F8Experts(torch.zeros(2, 4, 128, dtype=torch.uint8), torch.zeros(2, 4, 1), fp4.FP4_SCALES_1D, 4, 128)


@pytest.mark.parametrize("name,arguments", [
    ("fp8_gemm", lambda: dict(a=host_operand(), b=host_operand())),
    ("fp8_gemm", lambda: dict(b=host_operand(), a=host_operand())),
    ("fp8_expert_gemm", lambda: dict(x=host_operand(), w=host_stack(), plan=torch.zeros(3, dtype=torch.int32))),
    ("fp8_gated", lambda: dict(x=host_operand(), w=host_operand())),
    ("fp8_gated", lambda: dict(w=host_operand(), act="gelu", x=host_operand())),
    ("fp8_dequantize", lambda: dict(a=host_operand())),
])
def test_operands_by_keyword(name, arguments):
    """The call gets as far as the first operand's own check."""
    with pytest.raises(ValueError, match="device tensors"):
        getattr(fp4, name)(**arguments())


def test_a_missing_operand_is_named():
    with pytest.raises(TypeError, match="'x'"):
        fp4.fp8_gated(w=host_operand())
    with pytest.raises(TypeError, match="'a'"):
        fp4.fp8_gemm()


@pytest.mark.parametrize("dtype", [torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float8_e5m2fnuz, torch.float8_e8m0fnu,
                                   torch.int8, torch.bool])
def test_codes_of_another_type_are_refused(dtype):
    """One byte each, but not E4M3."""
    dev, q = torch.device("cpu"), torch.zeros(4, 256, dtype=torch.uint8).view(dtype)
    with pytest.raises(ValueError, match="codes must be"):
        fp8._operand(fp4.F8Tensor(q, torch.zeros(4, 2), fp4.FP4_SCALES_1D, 4, 200), "a", dev)
    with pytest.raises(ValueError, match="codes must be"):
        fp8._operand(fp4.F8Experts(q[None], torch.zeros(1, 4, 2), fp4.FP4_SCALES_1D, 4, 200), "w", dev, 1)


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.uint8])
def test_codes_of_the_right_types(dtype):
    q = torch.zeros(4, 256, dtype=torch.uint8).view(dtype)
    assert fp8._operand(fp4.F8Tensor(q, torch.zeros(4, 2), fp4.FP4_SCALES_1D, 4, 200), "a", torch.device("cpu")).rows == 4


def test_gated_grad_tiles_of_a_launch():
    """A launch holds fewer than 2^32 threads: 2^23 tiles of 128 x 128 are one too many for the float32 form's
    workgroups of 512, 2^24 for the bf16 form's of 256."""
    lib, p = _lib.load(), ctypes.c_void_p(4096)

    def views(dtype, rows, f):
        return lib.fp8_gated_grad(p, dtype, rows, f, f, p, 2 * f, 0, 0, p, p, p, p, None)
    assert views(1, 1 << 16, 1 << 21) == _lib.FP4_EUNSUPPORTED and "tiles" in lib.fp4_last_error().decode()
    assert views(0, 1 << 17, 1 << 21) == _lib.FP4_EUNSUPPORTED and "tiles" in lib.fp4_last_error().decode()
