"""Mixture-of-experts operators and weight-only FP4 products (include/fp4bs_experts.h).

A layer's forward pass is expert_sort -> expert_gather -> expert_linear (any number, with
activations between them) -> expert_combine; backward, expert_combine_grad -> expert_linear with
the transposed weights -> expert_gather_grad. `linear` is the product with one weight.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from . import QTensor, _dev_check, _in_dtype, _out_dtype, _stream


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


def expert_sort(ids: torch.Tensor, n_experts: int) -> ExpertPlan:
    """fp4_expert_sort: the plan of ids [tokens, topk] (int32 or int64; an id outside
    [0, n_experts) drops its slot)."""
    lib = _lib.load()
    _dev_check(ids)
    if ids.dim() != 2 or ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("ids must be a 2-D int32 or int64 tensor")
    if ids.shape[1] > 1 and ids.stride(1) != 1:
        raise ValueError("ids must have unit column stride")
    tokens, topk = ids.shape
    n, dev = tokens * topk, ids.device
    ws = ctypes.c_size_t()
    _lib.check(lib.fp4_expert_sort_workspace(tokens, topk, n_experts, ctypes.byref(ws)))
    order = torch.empty(n, dtype=torch.int32, device=dev)
    pos = torch.empty((tokens, topk), dtype=torch.int32, device=dev)
    offsets = torch.empty(n_experts + 1, dtype=torch.int32, device=dev)
    work = torch.empty(ws.value, dtype=torch.uint8, device=dev) if ws.value else None
    _lib.check(lib.fp4_expert_sort(ids.data_ptr(), int(ids.dtype == torch.int64), tokens, topk, _ld(ids), n_experts,
                                   order.data_ptr(), pos.data_ptr(), offsets.data_ptr(),
                                   work.data_ptr() if work is not None else None, ws.value, _stream()))
    return ExpertPlan(order, pos, offsets, tokens, topk, n_experts)


def _ld(t: torch.Tensor) -> int:
    """Row stride of a 2-D tensor; one row's stride says nothing and is taken as its width."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _rows_check(name: str, t: torch.Tensor, rows: int, width: int | None, dtype=None) -> None:
    if t.dim() != 2 or t.shape[0] != rows or (width is not None and t.shape[1] != width):
        raise ValueError(f"{name} must be [{rows}, {'hidden' if width is None else width}], got {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _out(out, rows, width, dtype, dev) -> torch.Tensor:
    if out is None:
        return torch.empty((rows, width), dtype=dtype, device=dev)
    _dev_check(out)
    _rows_check("out", out, rows, width, dtype)
    return out


def expert_gather(x: torch.Tensor, plan: ExpertPlan, out: torch.Tensor | None = None) -> torch.Tensor:
    """fp4_expert_gather: token rows [tokens, hidden] in expert order, [tokens * topk, hidden];
    dropped slots give zero rows."""
    lib = _lib.load()
    _dev_check(x)
    _rows_check("x", x, plan.tokens, None)
    out = _out(out, plan.tokens * plan.topk, x.shape[1], x.dtype, x.device)
    _lib.check(lib.fp4_expert_gather(x.data_ptr(), _in_dtype(x), plan.tokens, x.shape[1], _ld(x), plan.pos.data_ptr(),
                                     plan.topk, out.data_ptr(), _ld(out), _stream()))
    return out


def expert_gather_grad(dxs: torch.Tensor, plan: ExpertPlan, out: torch.Tensor | None = None) -> torch.Tensor:
    """fp4_expert_gather_grad: each token's sum [tokens, hidden] of its kept slots' rows."""
    lib = _lib.load()
    _dev_check(dxs)
    _rows_check("dxs", dxs, plan.tokens * plan.topk, None)
    out = _out(out, plan.tokens, dxs.shape[1], dxs.dtype, dxs.device)
    _lib.check(lib.fp4_expert_gather_grad(dxs.data_ptr(), _in_dtype(dxs), plan.tokens, dxs.shape[1], _ld(dxs),
                                          plan.pos.data_ptr(), plan.topk, out.data_ptr(), _ld(out), _stream()))
    return out


def expert_combine(ys: torch.Tensor, weights: torch.Tensor, plan: ExpertPlan,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """fp4_expert_combine: each token's weighted sum [tokens, hidden] of its kept slots' rows ys
    [tokens * topk, hidden]; weights float32 [tokens, topk]."""
    lib = _lib.load()
    _dev_check(ys, weights)
    _rows_check("ys", ys, plan.tokens * plan.topk, None)
    _rows_check("weights", weights, plan.tokens, plan.topk, torch.float32)
    out = _out(out, plan.tokens, ys.shape[1], ys.dtype, ys.device)
    _lib.check(lib.fp4_expert_combine(ys.data_ptr(), _in_dtype(ys), plan.tokens, ys.shape[1], _ld(ys),
                                      weights.data_ptr(), _ld(weights), plan.pos.data_ptr(), plan.topk,
                                      out.data_ptr(), _ld(out), _stream()))
    return out


def expert_combine_grad(dy: torch.Tensor, ys: torch.Tensor, weights: torch.Tensor, plan: ExpertPlan):
    """fp4_expert_combine_grad: (dys [tokens * topk, hidden] of ys's dtype, dweights float32
    [tokens, topk]) for dy [tokens, hidden]."""
    lib = _lib.load()
    _dev_check(dy, ys, weights)
    n, dev = plan.tokens * plan.topk, dy.device
    _rows_check("dy", dy, plan.tokens, None)
    _rows_check("ys", ys, n, dy.shape[1], dy.dtype)
    _rows_check("weights", weights, plan.tokens, plan.topk, torch.float32)
    dys = torch.empty((n, dy.shape[1]), dtype=dy.dtype, device=dev)
    dw = torch.empty((plan.tokens, plan.topk), dtype=torch.float32, device=dev)
    _lib.check(lib.fp4_expert_combine_grad(dy.data_ptr(), _in_dtype(dy), plan.tokens, dy.shape[1], _ld(dy),
                                           ys.data_ptr(), _ld(ys), weights.data_ptr(), _ld(weights),
                                           plan.pos.data_ptr(), plan.topk, dys.data_ptr(), _ld(dys), dw.data_ptr(),
                                           plan.topk, _stream()))
    return dys, dw


def _workspace(lib, rows: int, dt: int, op, n_experts: int, dev):
    ws = ctypes.c_size_t()
    _lib.check(lib.fp4_linear_workspace(rows, dt, ctypes.byref(op), n_experts, ctypes.byref(ws)))
    return (torch.empty(ws.value, dtype=torch.uint8, device=dev) if ws.value else None), ws.value


def linear(x: torch.Tensor, w: QTensor, out_dtype=None, out: torch.Tensor | None = None) -> torch.Tensor:
    """fp4_linear: x [rows, k] (bf16 or float32, not quantized) times the FP4 weight w [n, k]
    transposed, [rows, n] in out_dtype (x's by default). The transposed operand of a TILE2D weight
    gives the gradient dX = dY . W."""
    lib = _lib.load()
    _dev_check(x, w.q)
    if x.dim() != 2 or x.shape[1] != w.k or x.stride(1) != 1:
        raise ValueError(f"x must be [rows, {w.k}] with unit column stride, got {tuple(x.shape)}")
    dt = _in_dtype(x)
    out = _out(out, x.shape[0], w.rows, out_dtype or (x.dtype if out is None else out.dtype), x.device)
    op = w.operand()
    ws, nb = _workspace(lib, x.shape[0], dt, op, 0, x.device)
    _lib.check(lib.fp4_linear(x.data_ptr(), dt, x.shape[0], _ld(x), ctypes.byref(op), out.data_ptr(),
                              _out_dtype(out.dtype), _ld(out), ws.data_ptr() if nb else None, nb, _stream()))
    return out


def expert_linear(x: torch.Tensor, w: ExpertWeights, plan: ExpertPlan | torch.Tensor, out_dtype=None,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """fp4_expert_linear: rows x [rows, k] in expert order, each times its expert's weight
    transposed, [rows, n] in out_dtype (x's by default). plan: an ExpertPlan or its offsets (int32
    [n_experts + 1] on the device); rows past the last offset give zeros."""
    lib = _lib.load()
    offsets = plan.offsets if isinstance(plan, ExpertPlan) else plan
    _dev_check(x, w.q, offsets)
    if x.dim() != 2 or x.shape[1] != w.k or x.stride(1) != 1:
        raise ValueError(f"x must be [rows, {w.k}] with unit column stride, got {tuple(x.shape)}")
    if offsets.dtype != torch.int32 or offsets.shape != (w.n_experts + 1,) or not offsets.is_contiguous():
        raise ValueError(f"offsets must be a contiguous int32 tensor of {w.n_experts + 1} elements")
    dt = _in_dtype(x)
    out = _out(out, x.shape[0], w.rows, out_dtype or (x.dtype if out is None else out.dtype), x.device)
    op = w.operand()
    ws, nb = _workspace(lib, x.shape[0], dt, op, w.n_experts, x.device)
    _lib.check(lib.fp4_expert_linear(x.data_ptr(), dt, x.shape[0], _ld(x), ctypes.byref(op), w.n_experts,
                                     offsets.data_ptr(), out.data_ptr(), _out_dtype(out.dtype), _ld(out),
                                     ws.data_ptr() if nb else None, nb, _stream()))
    return out
