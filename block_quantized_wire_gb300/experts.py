"""The token side of a mixture-of-experts layer: sort, gather, combine and their gradients.

``sort`` orders the router's choices by expert; ``gather`` copies token rows into that
order; the experts work on their rows (``w4.matvec_w4_experts`` for 4-bit weights);
``combine`` brings the rows back, weighted and summed per token. ``combine_grad`` and
``gather_grad`` are the backward passes. As in ``codec``, outputs are caller-owned tensors
written in place, work is enqueued on the current stream (or ``stream``), and all
arithmetic runs in the library's kernels.

A slot is one choice of the router: slot ``t * top_k + j`` is token t's j-th expert. Its
place is its position in the order by expert. An id outside [0, n_experts) names an expert
that is not held here: the slot is dropped, and takes part in nothing.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from ._lib import check, load
from .codec import _stream

SORT_PARTS = 128  # BQ_SORT_PARTS
ROW_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # bq_row_type


class Plan(NamedTuple):
    """The places of a batch's slots, as ``sort`` writes them."""
    offsets: torch.Tensor    # int32 [n_experts + 1]: expert e's places are [offsets[e], offsets[e + 1])
    order: torch.Tensor      # int32 [tokens * top_k]: the slot at each place, -1 past the kept ones
    inverse: torch.Tensor    # int32 [tokens, top_k]: the place of each slot, -1 where dropped
    workspace: torch.Tensor  # int32 [SORT_PARTS, n_experts]: scratch of the sort


def empty_plan(tokens: int, top_k: int, n_experts: int, device="cuda") -> Plan:
    """The buffers that ``sort`` writes: ``sort(ids, n_experts, *empty_plan(...))``."""
    def ints(*shape):
        return torch.empty(shape, dtype=torch.int32, device=device)
    return Plan(ints(n_experts + 1), ints(tokens * top_k), ints(tokens, top_k), ints(SORT_PARTS, n_experts))


def _here(call: str, names: str, *tensors) -> int:
    """The current CUDA device, where the library launches: every tensor must live there."""
    cur = torch.cuda.current_device()
    for i, t in enumerate(tensors):
        if t is not None and t.get_device() != cur:
            where = t.device if t.is_cuda else "the CPU"
            raise ValueError(f"{call}: {names.split()[i]} is on {where}, but the current CUDA device is cuda:{cur}")
    return cur


def _on(stream, device: int) -> int:
    """The stream's handle; without one, the current stream's, which a decode step's many short
    calls read directly: a torch.cuda.Stream object would cost a third of such a call."""
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


def _flat(t: torch.Tensor, dtype: torch.dtype, name: str) -> int:
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def _row_type(t: torch.Tensor, name: str) -> int:
    kind = ROW_TYPES.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name}: expected bfloat16, float16 or float32, got {t.dtype}")
    return kind


def _rows(t: torch.Tensor, rows: int, cols: int, dtype: torch.dtype, name: str):
    """(pointer, leading dimension) of a row-major [rows, cols] view."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] != cols:
        raise ValueError(f"{name}: expected shape ({rows}, {cols}), got {tuple(shape)}")
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name}: expected unit column stride")
    return t.data_ptr(), ld if rows > 1 else cols


def sort(ids: torch.Tensor, n_experts: int, offsets: torch.Tensor, order: torch.Tensor, inverse: torch.Tensor,
         workspace: torch.Tensor, stream=None) -> None:
    """Router choices ids [tokens, top_k] (int32 or int64) -> a Plan's four buffers.
    Stable: within an expert, places go by slot (bq_expert_sort)."""
    if ids.dim() != 2:
        raise ValueError("sort: ids must be [tokens, top_k]")
    tokens, top_k = ids.shape
    wide = ids.dtype == torch.int64
    dev = _here("sort", "ids offsets order inverse workspace", ids, offsets, order, inverse, workspace)
    if (offsets.numel(), order.numel()) != (n_experts + 1, tokens * top_k) or inverse.shape != ids.shape:
        raise ValueError("sort: offsets must have n_experts + 1, order and inverse tokens * top_k values")
    if workspace.numel() < SORT_PARTS * n_experts:
        raise ValueError(f"sort: workspace needs {SORT_PARTS} * n_experts values")
    check("bq_expert_sort", load().bq_expert_sort(
        _flat(ids, torch.int64 if wide else torch.int32, "ids"), wide, tokens, top_k, n_experts,
        _flat(offsets, torch.int32, "offsets"), _flat(order, torch.int32, "order"),
        _flat(inverse, torch.int32, "inverse"), _flat(workspace, torch.int32, "workspace"), _on(stream, dev)))


def _plan_shape(inverse: torch.Tensor, call: str):
    if inverse.dim() != 2:
        raise ValueError(f"{call}: inverse must be [tokens, top_k]")
    return inverse.shape


def gather(x: torch.Tensor, inverse: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """Token rows x [tokens, hidden] -> out [tokens * top_k, hidden] by place, zeros past the
    kept places (bq_expert_gather)."""
    dev = _here("gather", "x inverse offsets out", x, inverse, offsets, out)
    tokens, top_k = _plan_shape(inverse, "gather")
    kind, hidden = _row_type(x, "x"), x.shape[-1]
    xp, ld_x = _rows(x, tokens, hidden, x.dtype, "x")
    op, ld_out = _rows(out, tokens * top_k, hidden, x.dtype, "out")
    check("bq_expert_gather", load().bq_expert_gather(
        xp, kind, tokens, hidden, ld_x, _flat(inverse, torch.int32, "inverse"), top_k,
        _flat(offsets, torch.int32, "offsets"), offsets.numel() - 1, op, ld_out, _on(stream, dev)))


def combine(y: torch.Tensor, weights: Optional[torch.Tensor], inverse: torch.Tensor, out: torch.Tensor,
            stream=None) -> None:
    """Expert rows y [tokens * top_k, hidden] -> out [tokens, hidden], row t the sum over j of
    weights[t, j] (float32; None: 1) times t's j-th expert row (bq_expert_combine)."""
    dev = _here("combine", "y weights inverse out", y, weights, inverse, out)
    tokens, top_k = _plan_shape(inverse, "combine")
    kind, hidden = _row_type(y, "y"), y.shape[-1]
    yp, ld_y = _rows(y, tokens * top_k, hidden, y.dtype, "y")
    op, ld_out = _rows(out, tokens, hidden, y.dtype, "out")
    if weights is not None and weights.shape != inverse.shape:
        raise ValueError("combine: weights must be [tokens, top_k]")
    check("bq_expert_combine", load().bq_expert_combine(
        yp, kind, ld_y, _flat(weights, torch.float32, "weights") if weights is not None else None,
        _flat(inverse, torch.int32, "inverse"), tokens, top_k, hidden, op, ld_out, _on(stream, dev)))


def gather_grad(dout: torch.Tensor, inverse: torch.Tensor, dx: torch.Tensor, stream=None) -> None:
    """The gradient of ``gather``: dx[t] = the sum of dout at t's places."""
    combine(dout, None, inverse, dx, stream)


def combine_grad(dout: torch.Tensor, y: torch.Tensor, weights: torch.Tensor, inverse: torch.Tensor,
                 offsets: torch.Tensor, dy: torch.Tensor, dweights: torch.Tensor, stream=None) -> None:
    """The gradients of ``combine``, in one pass: dy [tokens * top_k, hidden] by place (zeros
    past the kept places) and dweights [tokens, top_k] (bq_expert_combine_grad)."""
    dev = _here("combine_grad", "dout y weights inverse offsets dy dweights", dout, y, weights, inverse, offsets, dy,
                dweights)
    tokens, top_k = _plan_shape(inverse, "combine_grad")
    kind, hidden = _row_type(dout, "dout"), dout.shape[-1]
    dp, ld_d = _rows(dout, tokens, hidden, dout.dtype, "dout")
    yp, ld_y = _rows(y, tokens * top_k, hidden, dout.dtype, "y")
    gp, ld_g = _rows(dy, tokens * top_k, hidden, dout.dtype, "dy")
    if weights.shape != inverse.shape or dweights.shape != inverse.shape:
        raise ValueError("combine_grad: weights and dweights must be [tokens, top_k]")
    check("bq_expert_combine_grad", load().bq_expert_combine_grad(
        dp, kind, ld_d, yp, ld_y, _flat(weights, torch.float32, "weights"), _flat(inverse, torch.int32, "inverse"),
        _flat(offsets, torch.int32, "offsets"), offsets.numel() - 1, tokens, top_k, hidden, gp, ld_g,
        _flat(dweights, torch.float32, "dweights"), _on(stream, dev)))
