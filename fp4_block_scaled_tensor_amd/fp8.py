"""8-bit (E4M3) products with one scale to each block of 128, their quantizers and the gated feed-forward
projections (include/fp4bs_fp8.h).

A linear layer's training step: fp8_quantize_rowcol(x) and fp8_quantize(w, TILE2D), then fp8_gemm of the row
operands (forward), of dy's row operand and the weight's transposed one (dx), and of the two transposed
operands of dy and x (dw). A gated feed-forward block: fp8_gated, then fp8_gemm; backward, fp8_gated_grad
between the two layers' products. fp8_expert_gemm and fp8_gated with a plan take rows in expert order
(experts.py).
"""
from __future__ import annotations

import ctypes
import functools
import inspect
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import FP4_SCALES_1D, FP4_SCALES_2D, FP4_SCALES_2D_T, FP4_VIEW_COL, FP4_VIEW_ROW, FP4_VIEW_TILE2D
from .experts import ExpertPlan, _address, _current_device, _dtype, _ld, _matrix, _on_its_device, _stream_of

F8_SCALE_E8M0, F8_SCALE_F32 = _lib.FP8_SCALE_E8M0, _lib.FP8_SCALE_F32
BLOCK = 128
ACTIVATIONS = {"silu": _lib.FP8_ACT_SILU, "gelu": _lib.FP8_ACT_GELU, "gelu_tanh": _lib.FP8_ACT_GELU_TANH}
_SCALE_DTYPES = {F8_SCALE_E8M0: torch.float8_e8m0fnu, F8_SCALE_F32: torch.float32}
_BYTES = (torch.uint8, torch.float8_e8m0fnu)
_CODES = (torch.float8_e4m3fn, torch.uint8)


@dataclass
class F8Tensor:
    """An E4M3 operand [rows x k]: codes in rows of whole blocks (zeros past k) and their scales."""
    q: torch.Tensor          # float8_e4m3fn (or uint8) [rows, k in whole blocks of 128]
    s: torch.Tensor          # float8_e8m0fnu (or uint8) codes, or float32; shape by layout
    layout: int              # FP4_SCALES_*
    rows: int
    k: int


@dataclass
class F8Experts:
    """The weights of n_experts experts, each an operand [rows x k], stacked (fp8_stack)."""
    q: torch.Tensor          # [n_experts, rows, k in whole blocks of 128]
    s: torch.Tensor          # [n_experts, ...]
    layout: int
    rows: int
    k: int

    @property
    def n_experts(self) -> int:
        return self.q.shape[0]


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _scale_shape(layout: int, rows: int, k: int) -> tuple[int, int]:
    if layout == FP4_SCALES_1D:
        return rows, _blocks(k)
    grid = _blocks(rows), _blocks(k)
    return grid if layout == FP4_SCALES_2D else grid[::-1]


def fp8_stack(weights: list[F8Tensor]) -> F8Experts:
    """One F8Tensor per expert (same scale type, layout and sizes) as one stack."""
    if not weights:
        raise ValueError("no weights to stack")
    w = weights[0]
    if any((t.layout, t.rows, t.k, t.s.dtype) != (w.layout, w.rows, w.k, w.s.dtype) for t in weights):
        raise ValueError("the experts' weights must agree in scale type, layout and sizes")
    stack = lambda ts: torch.stack([t.view(torch.uint8) for t in ts]).view(ts[0].dtype)   # noqa: E731
    return F8Experts(stack([t.q for t in weights]), stack([t.s for t in weights]), w.layout, w.rows, w.k)


def _operand(a: F8Tensor | F8Experts, name: str, device: torch.device, n_experts: int = 0) -> _lib.F8Operand:
    """The C operand of a (one expert's of a stack) after its tensors are checked against its sizes."""
    q, s, many = a.q, a.s, n_experts or 1
    rows, cols = _scale_shape(a.layout, a.rows, a.k)
    if q.dtype not in _CODES or q.numel() != many * a.rows * _blocks(a.k) * BLOCK or not q.is_contiguous() or q.device != device:
        raise ValueError(f"{name}: codes must be a contiguous float8_e4m3fn (or uint8) tensor of "
                         f"{many * a.rows * _blocks(a.k) * BLOCK} bytes on {device}, got {q.dtype} {tuple(q.shape)} on {q.device}")
    if s.dtype in _BYTES:
        scale = F8_SCALE_E8M0
    elif s.dtype is torch.float32:
        scale = F8_SCALE_F32
    else:
        raise ValueError(f"{name}: scales must be float8_e8m0fnu (or uint8) or float32, got {s.dtype}")
    if s.numel() != many * rows * cols or not s.is_contiguous() or s.device != device:
        raise ValueError(f"{name}: scales must be a contiguous tensor of {many * rows * cols} elements on {device}, got "
                         f"{tuple(s.shape)} on {s.device}")
    return _lib.F8Operand(q.data_ptr(), s.data_ptr(), scale, a.layout, a.rows, a.k)


def _on_device_of(f):
    """f with the device of its first operand's codes made current (the library launches on the current one)."""
    first = next(iter(inspect.signature(f).parameters))

    @functools.wraps(f)
    def call(*args, **kwargs):
        a = args[0] if args else kwargs.get(first)
        if a is None:   # (f names the missing operand)
            return f(*args, **kwargs)
        if not a.q.is_cuda:
            raise ValueError("FP8 kernels take device tensors (the path has no CPU implementation)")
        device = a.q.get_device()
        if device == _current_device():
            return f(*args, **kwargs)
        with torch.cuda.device(device):
            return f(*args, **kwargs)
    return call


def _new(rows: int, k: int, scale: int, device) -> F8Tensor:
    """An operand with 1D scales to be written."""
    return F8Tensor(torch.empty(rows, _blocks(k) * BLOCK, dtype=torch.float8_e4m3fn, device=device),
                    torch.empty(rows, _blocks(k), dtype=_SCALE_DTYPES[scale], device=device), FP4_SCALES_1D, rows, k)


def _check_scale(scale: int) -> None:
    if scale not in _SCALE_DTYPES:
        raise ValueError(f"scale must be F8_SCALE_E8M0 or F8_SCALE_F32, got {scale}")


def _ptrs(t: F8Tensor | None):
    return (None, None) if t is None else (t.q.data_ptr(), t.s.data_ptr())


def _quantize(x: torch.Tensor, view: int, scale: int):
    lib = _lib.load()
    _check_scale(scale)
    rows, cols, ld = _matrix("x", x)
    dt, dev = _dtype(x, "x"), x.device
    row = col = None
    if view == FP4_VIEW_TILE2D:
        s = torch.empty(_blocks(rows), _blocks(cols), dtype=_SCALE_DTYPES[scale], device=dev)
        q = lambda r, k: torch.empty(r, _blocks(k) * BLOCK, dtype=torch.float8_e4m3fn, device=dev)   # noqa: E731
        row = F8Tensor(q(rows, cols), s, FP4_SCALES_2D, rows, cols)
        col = F8Tensor(q(cols, rows), s, FP4_SCALES_2D_T, cols, rows)
    else:
        if view != FP4_VIEW_COL:
            row = _new(rows, cols, scale, dev)
        if view != FP4_VIEW_ROW:
            col = _new(cols, rows, scale, dev)
    _lib.check(lib.fp8_quantize(x.data_ptr(), dt, rows, cols, ld, view, scale, *_ptrs(row), *_ptrs(col), _stream_of(x)))
    return row, col


@_on_its_device
def fp8_quantize(x: torch.Tensor, view: int = FP4_VIEW_ROW, scale: int = F8_SCALE_E8M0):
    """fp8_quantize: bf16 or float32 x [rows, cols] as an E4M3 operand. ROW: x with one scale to each 128 of
    a row. COL: x^T, one to each 128 of a column. TILE2D: the pair (x, x^T) sharing one scale to each
    128 x 128 tile."""
    if view not in (FP4_VIEW_ROW, FP4_VIEW_COL, FP4_VIEW_TILE2D):
        raise ValueError(f"view must be ROW, COL or TILE2D, got {view}")
    row, col = _quantize(x, view, scale)
    if view == FP4_VIEW_TILE2D:
        return row, col
    return col if row is None else row


@_on_its_device
def fp8_quantize_rowcol(x: torch.Tensor, scale: int = F8_SCALE_E8M0):
    """fp8_quantize: (ROW operand, COL operand) of x from one read; each equals its own call."""
    return _quantize(x, _lib.FP8_VIEW_ROWCOL, scale)


@_on_device_of
def fp8_dequantize(a: F8Tensor, out_dtype=torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """fp8_dequantize: the values [rows, k] of an operand, bfloat16 or float32."""
    lib = _lib.load()
    op = _operand(a, "a", a.q.device)
    if out is None:
        out, ld = torch.empty(a.rows, a.k, dtype=out_dtype, device=a.q.device), a.k
    else:
        ld = _ld("out", out, a.rows, a.k, out.dtype, a.q)
    _lib.check(lib.fp8_dequantize(ctypes.byref(op), out.data_ptr(), _dtype(out, "out"), ld, _stream_of(out)))
    return out


@functools.lru_cache(maxsize=4096)
def _workspace(rows: int, scale: int, layout: int, n: int, k: int, n_experts: int, gated: int, f32: int,
               device: int) -> int:
    """(device, the current one, is here for what is remembered: its compute units decide how K is split.)"""
    ws = ctypes.c_size_t()
    w = _lib.F8Operand(None, None, scale, layout, n, k)
    _lib.check(_lib.load().fp8_gemm_workspace(rows, ctypes.byref(w), n_experts, gated, f32,
                                               ctypes.byref(ws)))
    return ws.value


def _work(x: _lib.F8Operand, w: _lib.F8Operand, n_experts: int, gated: int, f32: bool, q: torch.Tensor):
    """The workspace of a product as a tensor to hold until its call has returned (or None), and its bytes."""
    n = _workspace(x.rows, x.scale, w.layout, w.rows, w.k, n_experts, gated, int(f32), q.get_device())
    return (torch.empty(n, dtype=torch.uint8, device=q.device) if n else None), n


def _offsets(plan, n_experts: int, x: F8Tensor) -> torch.Tensor:
    offsets = plan.offsets if isinstance(plan, ExpertPlan) else plan
    if (offsets.dtype is not torch.int32 or offsets.shape != (n_experts + 1,) or not offsets.is_contiguous()
            or offsets.device != x.q.device):
        raise ValueError(f"offsets must be a contiguous int32 tensor of {n_experts + 1} elements on {x.q.device}")
    if isinstance(plan, ExpertPlan) and x.rows != plan.tokens * plan.topk:
        raise ValueError(f"x must have the plan's {plan.tokens * plan.topk} rows (tokens * topk), got {x.rows}")
    return offsets


def _rows_out(name: str, out, rows: int, width: int, dtype, q: torch.Tensor):
    """An output [rows, width], made unless given, its type's code and row stride."""
    if out is None:
        out = torch.empty(rows, width, dtype=dtype, device=q.device)
        return out, _dtype(out, name), width
    return out, _dtype(out, name), _ld(name, out, rows, width, dtype or out.dtype, q)


@_on_device_of
def fp8_gemm(a: F8Tensor, b: F8Tensor, out_dtype=None, out: torch.Tensor | None = None) -> torch.Tensor:
    """fp8_gemm: a . b^T [a.rows, b.rows] in bfloat16 (the default) or float32, summed in float32. a has 1D
    scales; b any layout of the same scale type. A float32 result takes the bf16 matrix core, whose sums are
    as exact as its type and which has less than half the rate."""
    lib = _lib.load()
    x, w = _operand(a, "a", a.q.device), _operand(b, "b", a.q.device)
    if out is None and out_dtype is None:
        out_dtype = torch.bfloat16
    out, dt, ld = _rows_out("out", out, a.rows, b.rows, out_dtype, a.q)
    ws, nb = _work(x, w, 0, 0, dt, a.q)
    _lib.check(lib.fp8_gemm(ctypes.byref(x), ctypes.byref(w), out.data_ptr(), dt, ld, _address(ws), nb, _stream_of(a.q)))
    return out


@_on_device_of
def fp8_expert_gemm(x: F8Tensor, w: F8Experts, plan: ExpertPlan | torch.Tensor, out_dtype=None,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """fp8_expert_gemm: rows x in expert order, each times its expert's weight transposed. plan: an
    ExpertPlan or its offsets; rows past the last offset give zeros."""
    lib = _lib.load()
    n = w.n_experts
    offsets = _offsets(plan, n, x)
    a, b = _operand(x, "x", x.q.device), _operand(w, "w", x.q.device, n)
    if out is None and out_dtype is None:
        out_dtype = torch.bfloat16
    out, dt, ld = _rows_out("out", out, x.rows, w.rows, out_dtype, x.q)
    ws, nb = _work(a, b, n, 0, dt, x.q)
    _lib.check(lib.fp8_expert_gemm(ctypes.byref(a), ctypes.byref(b), n, offsets.data_ptr(), out.data_ptr(), dt, ld,
                                   _address(ws), nb, _stream_of(x.q)))
    return out


def _act(act: str) -> int:
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}, got {act!r}")
    return code


@_on_device_of
def fp8_gated(x: F8Tensor, w: F8Tensor | F8Experts, act: str = "silu", out_dtype=torch.bfloat16,
              save: torch.dtype | None = None, plan: ExpertPlan | torch.Tensor | None = None):
    """fp8_gated: (h, gu) with h = act(x . Wg^T) * (x . Wu^T) [rows, f] for w stacking gate and up projection
    [2 f, k]. out_dtype bfloat16 or float32, or float8_e4m3fn for h as the next product's operand (1D scales
    of x's type). save: the type in which the projections gu [rows, 2 f] are kept for the gradient, else None.
    With F8Experts and a plan: rows in expert order; rows past the last offset give zeros."""
    lib = _lib.load()
    kind = _act(act)
    experts = isinstance(w, F8Experts)
    if experts != (plan is not None):
        raise ValueError("a stack of experts takes a plan, one weight takes none")
    n = w.n_experts if experts else 0
    offsets = _offsets(plan, n, x) if experts else None
    a, b = _operand(x, "x", x.q.device), _operand(w, "w", x.q.device, n)
    if w.rows % 2:
        raise ValueError(f"w must stack gate and up projection, got {w.rows} rows")
    f = w.rows // 2
    ws, nb = _work(a, b, n, 2 if out_dtype is torch.float8_e4m3fn else 1, torch.float32 in (out_dtype, save), x.q)
    gu, gdt, ldgu = None, 0, 0
    if save is not None:
        gu, gdt, ldgu = _rows_out("gu", None, x.rows, w.rows, save, x.q)
    if out_dtype is torch.float8_e4m3fn:
        h = _new(x.rows, f, a.scale, x.q.device)
        hp, dt, ldh, hs = h.q.data_ptr(), _lib.FP8_OUT_E4M3, 0, h.s.data_ptr()
    else:
        h, dt, ldh = _rows_out("out", None, x.rows, f, out_dtype, x.q)
        hp, hs = h.data_ptr(), None
    _lib.check(lib.fp8_gated(ctypes.byref(a), ctypes.byref(b), n, None if offsets is None else offsets.data_ptr(), kind, hp,
                             dt, ldh, hs, _address(gu), gdt, ldgu, _address(ws), nb, _stream_of(x.q)))
    return h, gu


@_on_its_device
def gated_grad(dh: torch.Tensor, gu: torch.Tensor, act: str = "silu", out: torch.Tensor | None = None) -> torch.Tensor:
    """gated_grad: the gradient [rows, 2 f] of the projections gu [rows, 2 f] from dh [rows, f], both bfloat16 or
    both float32: dh * u * act'(g), then dh * act(g)."""
    lib = _lib.load()
    rows, f, lddh = _matrix("dh", dh)
    dt = _dtype(dh, "dh")
    ldgu = _ld("gu", gu, rows, 2 * f, dh.dtype, dh)
    out, _, ldo = _rows_out("out", out, rows, 2 * f, dh.dtype, dh)
    _lib.check(lib.gated_grad(dh.data_ptr(), dt, rows, f, lddh, gu.data_ptr(), ldgu, _act(act), out.data_ptr(), ldo,
                              _stream_of(dh)))
    return out


@_on_its_device
def fp8_gated_grad(dh: torch.Tensor, gu: torch.Tensor, act: str = "silu", scale: int = F8_SCALE_E8M0, row: bool = True,
                   col: bool = True):
    """fp8_gated_grad: the same gradient as the next products' operands, (ROW operand [rows x 2 f] for
    dx = dgu . W, COL operand [2 f x rows] for dw = dgu^T . x), None for one not asked for. f a multiple of 128."""
    lib = _lib.load()
    _check_scale(scale)
    rows, f, lddh = _matrix("dh", dh)
    dt = _dtype(dh, "dh")
    ldgu = _ld("gu", gu, rows, 2 * f, dh.dtype, dh)
    if not row and not col:
        raise ValueError("no view asked for")
    r = _new(rows, 2 * f, scale, dh.device) if row else None
    c = _new(2 * f, rows, scale, dh.device) if col else None
    _lib.check(lib.fp8_gated_grad(dh.data_ptr(), dt, rows, f, lddh, gu.data_ptr(), ldgu, _act(act), scale, *_ptrs(r),
                                  *_ptrs(c), _stream_of(dh)))
    return r, c
