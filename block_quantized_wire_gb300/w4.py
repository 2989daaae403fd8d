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
from .experts import _flat, _here, _on, _row_type, _rows


def _weights(call: str, q: torch.Tensor, scales: torch.Tensor, x: torch.Tensor, dims: int):
    """(n, k, group, scale type) of a weight matrix; the checks that need the tensors."""
    if q.dtype != torch.uint8:
        raise TypeError(f"{call}: q must be uint8, got {q.dtype}")
    if q.dim() != dims or scales.shape[:-1] != q.shape[:-1]:
        raise ValueError(f"{call}: q and scales must have {dims} dimensions, alike but the last")
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"{call}: x must be bfloat16 or float16, got {x.dtype}")
    if scales.dtype not in (x.dtype, torch.float32):
        raise TypeError(f"{call}: scales must be {x.dtype} or float32, got {scales.dtype}")
    n, k = q.shape[-2], 2 * q.shape[-1]
    groups = scales.shape[-1]
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError(f"{call}: x must be [rows, {k}]")
    group = k // groups if groups else 32
    if group not in (32, 64, 128) or groups * group != k:
        raise ValueError(f"{call}: {k} columns with {groups} scales a row: a scale covers 32, 64 or 128 columns")
    if (q.shape[-1] > 1 and q.stride(-1) != 1) or (groups > 1 and scales.stride(-1) != 1):
        raise ValueError(f"{call}: q and scales must have unit column stride")
    return n, k, group, _row_type(scales, "scales")


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
    if group not in (32, 64, 128) or groups * group != k:
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
    (bq_matvec_w4). Any number of rows; made for up to 32."""
    dev = _here("matvec_w4", "x q scales out", x, q, scales, out)
    n, k, group, s_kind = _weights("matvec_w4", q, scales, x, 2)
    rows = x.shape[0]
    xp, ld_x = _rows(x, rows, k, x.dtype, "x")
    op, ld_out = _rows(out, rows, n, x.dtype, "out")
    one = n <= 1
    check("bq_matvec_w4", load().bq_matvec_w4(
        xp, _row_type(x, "x"), rows, k, ld_x, q.data_ptr(), n, k // 2 if one else q.stride(0), scales.data_ptr(),
        s_kind, group, k // group if one else scales.stride(0), op, ld_out, _on(stream, dev)))


def matvec_w4_experts(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, offsets: torch.Tensor,
                      out: torch.Tensor, order: Optional[torch.Tensor] = None, top_k: int = 1, stream=None) -> None:
    """Each place's row times its own expert's weights: q [n_experts, n, k/2], out
    [slots, n], zeros past the kept places (bq_matvec_w4_experts). With ``order`` (of
    ``experts.sort``) place p takes row order[p] // top_k of x, the tokens' rows; without it
    x [slots, k] is already by place."""
    dev = _here("matvec_w4_experts", "x q scales offsets out order", x, q, scales, offsets, out, order)
    n, k, group, s_kind = _weights("matvec_w4_experts", q, scales, x, 3)
    n_experts = q.shape[0]
    slots, x_rows = out.shape[0], x.shape[0]
    if offsets.numel() != n_experts + 1:
        raise ValueError("matvec_w4_experts: offsets must have n_experts + 1 values")
    if order is not None and order.numel() != slots:
        raise ValueError("matvec_w4_experts: order must have one value for each row of out")
    xp, ld_x = _rows(x, x_rows, k, x.dtype, "x")
    op, ld_out = _rows(out, slots, n, x.dtype, "out")
    one = n <= 1
    check("bq_matvec_w4_experts", load().bq_matvec_w4_experts(
        xp, _row_type(x, "x"), x_rows, k, ld_x, q.data_ptr(), n, k // 2 if one else q.stride(1), q.stride(0),
        scales.data_ptr(), s_kind, group, k // group if one else scales.stride(1), scales.stride(0),
        _flat(offsets, torch.int32, "offsets"), n_experts, _flat(order, torch.int32, "order") if order is not None
        else None, top_k, slots, op, ld_out, _on(stream, dev)))
