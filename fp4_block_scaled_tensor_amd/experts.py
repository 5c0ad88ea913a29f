"""Mixture-of-experts operators and weight-only FP4 products (include/fp4bs_experts.h).

A layer's forward pass is expert_sort -> expert_gather -> expert_linear (any number, with
activations between them) -> expert_combine; backward, expert_combine_grad -> expert_linear with
the transposed weights -> expert_gather_grad. `linear` is the product with one weight.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
from dataclasses import dataclass

import torch

from . import _lib
from . import QTensor, _dev_check


@dataclass
class ExpertPlan:
    """Where each (token, choice) slot goes when the slots are sorted by expert (expert_sort)."""
    order: torch.Tensor      # int32 [tokens * topk]: slot of each position
    pos: torch.Tensor        # int32 [tokens, topk]: position of each slot, ~position if it is dropped
    offsets: torch.Tensor    # int32 [n_experts + 1]: first position of each expert; last: kept slots
    tokens: int
    topk: int
    n_experts: int


@dataclass
class ExpertWeights:
    """FP4 weights of n_experts experts, each [rows x k], stacked (stack_experts)."""
    q: torch.Tensor          # uint8 [n_experts, rows, k // 2]
    s: torch.Tensor          # uint8 scale codes [n_experts, ...]
    g: torch.Tensor          # float32 [n_experts, floats of one expert]
    fmt: int
    block: int
    layout: int              # FP4_SCALES_*
    rows: int
    k: int
    g_stripe: int = 0

    @property
    def n_experts(self) -> int:
        return self.q.shape[0]

    def operand(self) -> _lib.Operand:
        return _lib.Operand(self.q.data_ptr(), self.s.data_ptr(), self.g.data_ptr(), self.fmt, self.block,
                            self.layout, self.g_stripe, self.rows, self.k)


def stack_experts(weights: list[QTensor]) -> ExpertWeights:
    """One QTensor per expert (same format, block, scale layout and sizes) as one stack. For a
    TILE2D quantization stack the forward operands, and the transposed ones for the gradient."""
    if not weights:
        raise ValueError("no weights to stack")
    w = weights[0]
    key = lambda t: (t.fmt, t.block, t.layout, t.rows, t.k, t.g_stripe, t.g.numel())   # noqa: E731
    if any(key(t) != key(w) for t in weights):
        raise ValueError("the experts' weights must agree in format, block, scale layout and sizes")
    return ExpertWeights(torch.stack([t.q for t in weights]), torch.stack([t.s for t in weights]),
                         torch.stack([t.g for t in weights]), w.fmt, w.block, w.layout, w.rows, w.k, w.g_stripe)


# The calls below are short next to their launches, so the checks read each property once and the
# workspace sizes, which depend on nothing but the sizes, are remembered by them.
_DTYPES = {torch.bfloat16: _lib.FP4_IN_BF16, torch.float32: _lib.FP4_IN_FP32}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_of(t: torch.Tensor) -> int:
    """The current stream of t's device."""
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _dtype(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return code


def _on_its_device(f):
    """f with the device of its first tensor made current: the library launches on the current one."""
    first = next(iter(inspect.signature(f).parameters))

    @functools.wraps(f)
    def call(*args, **kwargs):
        t = args[0] if args else kwargs.get(first)
        device = -1 if t is None else t.get_device()
        if device < 0 or device == _current_device():   # (f refuses a missing or host tensor)
            return f(*args, **kwargs)
        with torch.cuda.device(device):
            return f(*args, **kwargs)
    return call


def _matrix(name: str, t: torch.Tensor) -> tuple[int, int, int]:
    """Checks a device matrix with unit column stride, a call's first; its rows, width and row stride (one
    row's says nothing and is taken as its width)."""
    if not t.is_cuda:
        _dev_check(t)
    shape, stride = t.shape, t.stride()
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(shape)}")
    rows, width = shape
    if width > 1 and stride[1] != 1:
        raise ValueError(f"{name} must have unit column stride")
    return rows, width, stride[0] if rows > 1 else width


def _ld(name: str, t: torch.Tensor, rows: int, width: int, dtype: torch.dtype, like: torch.Tensor) -> int:
    """Checks a further matrix of a call, [rows, width] of dtype on the device of its first; its row stride."""
    if t.device != like.device:
        raise ValueError(f"{name} must be on {like.device}, got {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    got, wide, ld = _matrix(name, t)
    if got != rows or wide != width:
        raise _mismatch(name, t, rows, width)
    return ld


def _mismatch(name: str, t: torch.Tensor, rows: int, width: int) -> ValueError:
    return ValueError(f"{name} must be [{rows}, {width}], got {tuple(t.shape)}")


def _pos(plan: ExpertPlan, like: torch.Tensor) -> int:
    """The address of a plan's positions, which the kernels read as packed int32 on like's device
    (the rows' own checks do not cover them, and plans are also built by callers)."""
    pos = plan.pos
    if (pos.dtype is not torch.int32 or pos.numel() != plan.tokens * plan.topk or not pos.is_contiguous()
            or pos.device != like.device):
        raise ValueError(f"plan.pos must be a contiguous int32 tensor [{plan.tokens}, {plan.topk}] on {like.device}, got "
                         f"{pos.dtype} {tuple(pos.shape)} on {pos.device}")
    return pos.data_ptr()


@functools.lru_cache(maxsize=4096)
def _sort_workspace(tokens: int, topk: int, n_experts: int) -> int:
    ws = ctypes.c_size_t()
    _lib.check(_lib.load().fp4_expert_sort_workspace(tokens, topk, n_experts, ctypes.byref(ws)))
    return ws.value


@functools.lru_cache(maxsize=4096)
def _linear_workspace(rows: int, dtype: int, fmt: int, block: int, layout: int, g_stripe: int, n: int, k: int,
                      n_experts: int, device: int = -1) -> int:
    """(device, the current one, is here for what is remembered: its compute units decide how K is split.)"""
    ws = ctypes.c_size_t()
    op = _lib.Operand(None, None, None, fmt, block, layout, g_stripe, n, k)
    _lib.check(_lib.load().fp4_linear_workspace(rows, dtype, ctypes.byref(op), n_experts, ctypes.byref(ws)))
    return ws.value


def _address(workspace: torch.Tensor | None) -> int | None:
    """A workspace's address. The caller keeps the tensor in a local until the library call has
    returned: only then is everything enqueued that uses it, and a block that is dropped before may
    be given to another thread (the call releases the interpreter lock) or be unmapped."""
    return None if workspace is None else workspace.data_ptr()


@_on_its_device
def expert_sort(ids: torch.Tensor, n_experts: int) -> ExpertPlan:
    """fp4_expert_sort: the plan of ids [tokens, topk] (int32 or int64; an id outside
    [0, n_experts) drops its slot)."""
    lib = _lib.load()
    if ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("ids must be a 2-D int32 or int64 tensor")
    tokens, topk, ld = _matrix("ids", ids)
    n, dev = tokens * topk, ids.device
    nb = _sort_workspace(tokens, topk, n_experts)
    order = torch.empty(n, dtype=torch.int32, device=dev)
    pos = torch.empty(tokens, topk, dtype=torch.int32, device=dev)
    offsets = torch.empty(n_experts + 1, dtype=torch.int32, device=dev)
    work = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
    _lib.check(lib.fp4_expert_sort(ids.data_ptr(), int(ids.dtype is torch.int64), tokens, topk, ld, n_experts,
                                   order.data_ptr(), pos.data_ptr(), offsets.data_ptr(), _address(work), nb,
                                   _stream_of(ids)))
    return ExpertPlan(order, pos, offsets, tokens, topk, n_experts)


@_on_its_device
def expert_gather(x: torch.Tensor, plan: ExpertPlan, out: torch.Tensor | None = None) -> torch.Tensor:
    """fp4_expert_gather: token rows [tokens, hidden] in expert order, [tokens * topk, hidden];
    dropped slots give zero rows."""
    lib = _lib.load()
    (rows, h, ldx), n = _matrix("x", x), plan.tokens * plan.topk
    if rows != plan.tokens:
        raise _mismatch("x", x, plan.tokens, h)
    dt = _dtype(x, "x")
    if out is None:
        out, ldo = x.new_empty(n, h), h
    else:
        ldo = _ld("out", out, n, h, x.dtype, x)
    _lib.check(lib.fp4_expert_gather(x.data_ptr(), dt, plan.tokens, h, ldx, _pos(plan, x), plan.topk,
                                     out.data_ptr(), ldo, _stream_of(x)))
    return out


@_on_its_device
def expert_gather_grad(dxs: torch.Tensor, plan: ExpertPlan, out: torch.Tensor | None = None) -> torch.Tensor:
    """fp4_expert_gather_grad: each token's sum [tokens, hidden] of its kept slots' rows."""
    lib = _lib.load()
    rows, h, ld = _matrix("dxs", dxs)
    if rows != plan.tokens * plan.topk:
        raise _mismatch("dxs", dxs, plan.tokens * plan.topk, h)
    dt = _dtype(dxs, "dxs")
    if out is None:
        out, ldo = dxs.new_empty(plan.tokens, h), h
    else:
        ldo = _ld("out", out, plan.tokens, h, dxs.dtype, dxs)
    _lib.check(lib.fp4_expert_gather_grad(dxs.data_ptr(), dt, plan.tokens, h, ld, _pos(plan, dxs), plan.topk,
                                          out.data_ptr(), ldo, _stream_of(dxs)))
    return out


@_on_its_device
def expert_combine(ys: torch.Tensor, weights: torch.Tensor, plan: ExpertPlan,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """fp4_expert_combine: each token's weighted sum [tokens, hidden] of its kept slots' rows ys
    [tokens * topk, hidden]; weights float32 [tokens, topk]."""
    lib = _lib.load()
    rows, h, ld = _matrix("ys", ys)
    if rows != plan.tokens * plan.topk:
        raise _mismatch("ys", ys, plan.tokens * plan.topk, h)
    ldw = _ld("weights", weights, plan.tokens, plan.topk, torch.float32, ys)
    dt = _dtype(ys, "ys")
    if out is None:
        out, ldo = ys.new_empty(plan.tokens, h), h
    else:
        ldo = _ld("out", out, plan.tokens, h, ys.dtype, ys)
    _lib.check(lib.fp4_expert_combine(ys.data_ptr(), dt, plan.tokens, h, ld, weights.data_ptr(), ldw,
                                      _pos(plan, ys), plan.topk, out.data_ptr(), ldo, _stream_of(ys)))
    return out


@_on_its_device
def expert_combine_grad(dy: torch.Tensor, ys: torch.Tensor, weights: torch.Tensor, plan: ExpertPlan):
    """fp4_expert_combine_grad: (dys [tokens * topk, hidden] of ys's dtype, dweights float32
    [tokens, topk]) for dy [tokens, hidden]."""
    lib = _lib.load()
    (rows, h, lddy), n = _matrix("dy", dy), plan.tokens * plan.topk
    if rows != plan.tokens:
        raise _mismatch("dy", dy, plan.tokens, h)
    ldys = _ld("ys", ys, n, h, dy.dtype, dy)
    ldw = _ld("weights", weights, plan.tokens, plan.topk, torch.float32, dy)
    dt = _dtype(dy, "dy")
    dys = dy.new_empty(n, h)
    dw = weights.new_empty(plan.tokens, plan.topk)
    _lib.check(lib.fp4_expert_combine_grad(dy.data_ptr(), dt, plan.tokens, h, lddy, ys.data_ptr(), ldys,
                                           weights.data_ptr(), ldw, _pos(plan, dy), plan.topk, dys.data_ptr(), h,
                                           dw.data_ptr(), plan.topk, _stream_of(dy)))
    return dys, dw


@functools.lru_cache(maxsize=4096)
def _weight_bytes(rows: int, k: int, block: int, layout: int, g_stripe: int) -> tuple[int, int, int]:
    """Bytes of one weight's payload, scale codes and g."""
    scales = rows * (k // block) if layout == _lib.FP4_SCALES_1D else (rows // 16) * (k // 16)
    return rows * (k // 2), scales, 4 * max(1, -(-rows // g_stripe) if g_stripe else 1)


def _check_weight(w: QTensor | ExpertWeights, n_experts: int, like: torch.Tensor) -> None:
    """The buffers of a weight (n_experts 0) or of a stack against its sizes: packed on like's device, and
    a stack's experts without a gap."""
    q, s, g, dev, many = w.q, w.s, w.g, like.device, n_experts or 1
    nq, ns, ng = _weight_bytes(w.rows, w.k, w.block, w.layout, w.g_stripe)
    if not ((q.nbytes == nq * many or (q.nbytes > nq and not n_experts)) and q.is_contiguous() and q.device == dev
            and q.element_size() == 1):
        bad, t, size = "payload", q, nq
    elif not ((s.nbytes == ns * many or (s.nbytes > ns and not n_experts)) and s.is_contiguous() and s.device == dev
              and s.element_size() == 1):
        bad, t, size = "scales", s, ns
    elif not ((g.nbytes == ng * many or (g.nbytes > ng and not n_experts) or (g.nbytes == 0 and not w.g_stripe))   # none: 1
              and g.is_contiguous() and g.device == dev and g.dtype is torch.float32):
        bad, t, size = "g", g, ng
    else:
        return
    raise ValueError(f"the weight's {bad} must be a contiguous {'float32' if t is g else 'uint8'} tensor of "
                     f"{size * many} bytes on {dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _product(x, w, rows, k, n_experts, out_dtype, out):
    """What linear and expert_linear share: checks, output, workspace (a tensor to hold, see _address)."""
    if k != w.k:
        raise _mismatch("x", x, rows, w.k)
    dt = odt = _dtype(x, "x")
    if out is None:
        ldo = w.rows
        if out_dtype is None:
            out = x.new_empty(rows, ldo)
        else:
            out = x.new_empty((rows, ldo), dtype=out_dtype)
            odt = _dtype(out, "out")
    else:
        ldo = _ld("out", out, rows, w.rows, out_dtype or out.dtype, x)
        odt = _dtype(out, "out")
    nb = _linear_workspace(rows, dt, w.fmt, w.block, w.layout, w.g_stripe, w.rows, w.k, n_experts, x.get_device())
    _check_weight(w, n_experts, x)
    ws = x.new_empty(nb, dtype=torch.uint8) if nb else None
    return dt, out, ldo, odt, ws, nb


@_on_its_device
def linear(x: torch.Tensor, w: QTensor, out_dtype=None, out: torch.Tensor | None = None) -> torch.Tensor:
    """fp4_linear: x [rows, k] (bf16 or float32, not quantized) times the FP4 weight w [n, k]
    transposed, [rows, n] in out_dtype (x's by default). The transposed operand of a TILE2D weight
    gives the gradient dX = dY . W."""
    lib = _lib.load()
    rows, k, ldx = _matrix("x", x)
    dt, out, ldo, odt, ws, nb = _product(x, w, rows, k, 0, out_dtype, out)
    op = w.operand()
    _lib.check(lib.fp4_linear(x.data_ptr(), dt, rows, ldx, ctypes.byref(op), out.data_ptr(), odt, ldo, _address(ws),
                              nb, _stream_of(x)))
    return out


@_on_its_device
def expert_linear(x: torch.Tensor, w: ExpertWeights, plan: ExpertPlan | torch.Tensor, out_dtype=None,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """fp4_expert_linear: rows x [rows, k] in expert order, each times its expert's weight
    transposed, [rows, n] in out_dtype (x's by default). plan: an ExpertPlan or its offsets (int32
    [n_experts + 1] on x's device); rows past the last offset give zeros. With an ExpertPlan x has its
    tokens * topk rows, with offsets any number of at least the last one."""
    lib = _lib.load()
    offsets = plan.offsets if isinstance(plan, ExpertPlan) else plan
    experts = w.n_experts
    rows, k, ldx = _matrix("x", x)
    if (offsets.dtype is not torch.int32 or offsets.shape != (experts + 1,) or not offsets.is_contiguous()
            or offsets.device != x.device):
        raise ValueError(f"offsets must be a contiguous int32 tensor of {experts + 1} elements on {x.device}")
    if isinstance(plan, ExpertPlan) and rows != plan.tokens * plan.topk:
        raise ValueError(f"x must have the plan's {plan.tokens * plan.topk} rows (tokens * topk), got {rows}")
    dt, out, ldo, odt, ws, nb = _product(x, w, rows, k, experts, out_dtype, out)
    op = w.operand()
    _lib.check(lib.fp4_expert_linear(x.data_ptr(), dt, rows, ldx, ctypes.byref(op), experts, offsets.data_ptr(),
                                     out.data_ptr(), odt, ldo, _address(ws), nb, _stream_of(x)))
    return out
