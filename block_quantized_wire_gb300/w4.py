"""Products of a few rows with 4-bit weights and group scales: the decode step's linear layers.

A weight matrix [n, k] is ``q`` (uint8 [n, k/2]: two signed 4-bit codes a byte, the even
column in the low half) and ``scales`` ([n, k/group], the type of the activations or
float32, group 32, 64 or 128): weight = code * scale. Experts' weights have a leading
dimension more. ``x`` and ``q`` rows start on 16-byte boundaries.
"""
from __future__ import annotations

from typing import Optional

import torch

from ._lib import check, load
from .experts import ROW_TYPES, _flat, _here, _on, _row_type, _rows


GROUPS = (32, 64, 128)


def _weights(call: str, q: torch.Tensor, scales: torch.Tensor, x: torch.Tensor, dims: int):
    """(n, k, group, x type, scale type, row strides of q and scales) of a weight matrix; the
    checks that need the tensors."""
    x_type, s_type, q_shape, s_shape, x_shape = x.dtype, scales.dtype, q.shape, scales.shape, x.shape
    if q.dtype is not torch.uint8:
        raise TypeError(f"{call}: q must be uint8, got {q.dtype}")
    if len(q_shape) != dims or q_shape[:-1] != s_shape[:-1]:
        raise ValueError(f"{call}: q and scales must have {dims} dimensions, alike but the last")
    if x_type is not torch.bfloat16 and x_type is not torch.float16:
        raise TypeError(f"{call}: x must be bfloat16 or float16, got {x_type}")
    if s_type is not x_type and s_type is not torch.float32:
        raise TypeError(f"{call}: scales must be {x_type} or float32, got {s_type}")
    n, half, groups = q_shape[-2], q_shape[-1], s_shape[-1]
    k = 2 * half
    if len(x_shape) != 2 or x_shape[1] != k:
        raise ValueError(f"{call}: x must be [rows, {k}]")
    group = k // groups if groups else 32
    if group not in GROUPS or groups * group != k:
        raise ValueError(f"{call}: {k} columns with {groups} scales a row: a scale covers 32, 64 or 128 columns")
    q_stride, s_stride = q.stride(), scales.stride()
    if (q_stride[-1] != 1 and half > 1) or (s_stride[-1] != 1 and groups > 1):
        raise ValueError(f"{call}: q and scales must have unit column stride")
    ld_q, ld_s = (q_stride[-2], s_stride[-2]) if n > 1 else (half, groups)
    return n, k, group, ROW_TYPES[x_type], ROW_TYPES[s_type], ld_q, ld_s


def empty_w4(n: int, k: int, group: int, scale_dtype=torch.bfloat16, device="cuda", lead=()):
    """(q, scales) of a weight matrix [n, k], or of several with the leading dimensions `lead`."""
    return (torch.empty((*lead, n, k // 2), dtype=torch.uint8, device=device),
            torch.empty((*lead, n, k // group), dtype=scale_dtype, device=device))


def quant_w4(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """Weights x [n, k] or [n_experts, n, k] (bfloat16, float16 or float32) -> codes q and group
    scales: amax / 7 per group, the nearest code (bq_quant_w4). Leading dimensions must be
    contiguous with the rows."""
    dev = _here("quant_w4", "x q scales", x, q, scales)
    if q.dtype != torch.uint8:
        raise TypeError(f"quant_w4: q must be uint8, got {q.dtype}")
    if x.dim() < 2 or q.shape != (*x.shape[:-1], x.shape[-1] // 2) or scales.shape[:-1] != x.shape[:-1]:
        raise ValueError("quant_w4: q must be [..., n, k / 2] and scales [..., n, k / group]")
    k, groups = x.shape[-1], scales.shape[-1]
    group = k // groups if groups else 32
    if group not in GROUPS or groups * group != k:
        raise ValueError(f"quant_w4: {k} columns with {groups} scales a row: a scale covers 32, 64 or 128 columns")
    n = x.numel() // k if k else 0
    flat = [t.view(n, t.shape[-1]) if n else t for t in (x, q, scales)]
    xp, ld_x = _rows(flat[0], n, k, x.dtype, "x") if n else (None, k)
    qp, ld_q = _rows(flat[1], n, k // 2, torch.uint8, "q") if n else (None, k)
    sp, ld_s = _rows(flat[2], n, groups, scales.dtype, "scales") if n else (None, k)
    check("bq_quant_w4", load().bq_quant_w4(xp, _row_type(x, "x"), n, k, ld_x, group, qp, ld_q, sp,
                                            _row_type(scales, "scales"), ld_s, _on(stream, dev)))


def matvec_w4(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """x [rows, k] times the weights [n, k] transposed -> out [rows, n] of x's type
    (bq_matvec_w4). Any number of rows; made for up to 16, and 16 at a time."""
    dev = _here("matvec_w4", "x q scales out", x, q, scales, out)
    n, k, group, kind, s_kind, ld_q, ld_s = _weights("matvec_w4", q, scales, x, 2)
    rows = x.shape[0]
    xp, ld_x = _rows(x, rows, k, x.dtype, "x")
    op, ld_out = _rows(out, rows, n, x.dtype, "out")
    check("bq_matvec_w4", load().bq_matvec_w4(xp, kind, rows, k, ld_x, q.data_ptr(), n, ld_q, scales.data_ptr(),
                                              s_kind, group, ld_s, op, ld_out, _on(stream, dev)))


def matvec_w4_experts(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, offsets: torch.Tensor,
                      out: torch.Tensor, order: Optional[torch.Tensor] = None, top_k: int = 1, stream=None) -> None:
    """Each place's row times its own expert's weights: q [n_experts, n, k/2], out
    [slots, n], zeros past the kept places (bq_matvec_w4_experts). With ``order`` (of
    ``experts.sort``) place p takes row order[p] // top_k of x, the tokens' rows; without it
    x [slots, k] is already by place."""
    dev = _here("matvec_w4_experts", "x q scales offsets out order", x, q, scales, offsets, out, order)
    n, k, group, kind, s_kind, ld_q, ld_s = _weights("matvec_w4_experts", q, scales, x, 3)
    n_experts = q.shape[0]
    slots, x_rows = out.shape[0], x.shape[0]
    if offsets.numel() != n_experts + 1:
        raise ValueError("matvec_w4_experts: offsets must have n_experts + 1 values")
    if order is not None and order.numel() != slots:
        raise ValueError("matvec_w4_experts: order must have one value for each row of out")
    xp, ld_x = _rows(x, x_rows, k, x.dtype, "x")
    op, ld_out = _rows(out, slots, n, x.dtype, "out")
    check("bq_matvec_w4_experts", load().bq_matvec_w4_experts(
        xp, kind, x_rows, k, ld_x, q.data_ptr(), n, ld_q, q.stride(0), scales.data_ptr(), s_kind, group, ld_s,
        scales.stride(0), _flat(offsets, torch.int32, "offsets"), n_experts,
        _flat(order, torch.int32, "order") if order is not None else None, top_k, slots, op, ld_out,
        _on(stream, dev)))
