"""A key-value cache in 4 bits, in pages: written a row at a time, read back, and attended over.

A row is one head of one token, of keys or of values: signed 4-bit codes (two a byte, the even
column in the low half, as in ``w4``) and a (scale, offset) pair of 16-bit values for each group of
32, 64 or 128 columns; a code stands for ``code * scale + offset``. A slot is ``page * tokens per
page + place``. As in ``codec``, outputs are caller-owned tensors written in place, work is enqueued
on the current stream (or ``stream``), and all arithmetic runs in the library's kernels.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._lib import Kv4Cache as _Kv4Cache
from ._lib import check, load
from .experts import ROW_TYPES, _flat, _here, _on
from .w4 import GROUPS

HEAD_DIMS = (64, 128, 192, 256)


class Cache:
    """The tensors of a cache and what a call needs to know of them, checked once.

    ``k`` and ``v`` uint8 [pages, heads, page, head_dim / 2]: the codes; ``k_scales`` and
    ``v_scales`` bfloat16 or float16 [pages, heads, page, head_dim / group, 2]: the (scale, offset)
    pairs. Any strides that keep rows contiguous and apart (a view that has tokens before heads, or
    keys and values of a page in one block, works), the same for keys and values; rows of codes
    start on 16-byte boundaries, rows of pairs on the largest power of two that divides their
    bytes, at most 16. 1 to 1024 heads, 1 to 65536 tokens a page. The tensors must stay where they
    are while the object is in use."""

    def __init__(self, k: torch.Tensor, k_scales: torch.Tensor, v: torch.Tensor, v_scales: torch.Tensor):
        dtype = k_scales.dtype
        if k.dtype is not torch.uint8 or v.dtype is not torch.uint8:
            raise TypeError(f"Cache: codes must be uint8, got {k.dtype} and {v.dtype}")
        if dtype not in (torch.bfloat16, torch.float16) or v_scales.dtype is not dtype:
            raise TypeError(f"Cache: scales must be bfloat16 or float16, both alike, got {dtype} and {v_scales.dtype}")
        if k.dim() != 4 or k_scales.dim() != 5 or k_scales.shape[:3] != k.shape[:3] or k_scales.shape[4] != 2:
            raise ValueError("Cache: codes must be [pages, heads, page, head_dim / 2], scales [pages, heads, page, "
                             "head_dim / group, 2]")
        if k.shape != v.shape or k_scales.shape != v_scales.shape:
            raise ValueError("Cache: keys and values must have the same shapes")
        pages, heads, page, half = k.shape
        head_dim, groups = 2 * half, k_scales.shape[3]
        group = head_dim // groups if groups else 0
        if head_dim not in HEAD_DIMS or group not in GROUPS or groups * group != head_dim:
            raise ValueError(f"Cache: head_dim {head_dim} with {groups} scales a row: head_dim must be 64, 128, 192 or "
                             "256, and a scale covers 32, 64 or 128 columns")
        if not 1 <= heads <= 1024 or not 1 <= page <= 65536:  # BQ_KV4_MAX_HEADS, BQ_KV4_MAX_PAGE
            raise ValueError(f"Cache: 1 to 1024 heads and 1 to 65536 tokens a page, got {heads} and {page}")
        for t, last in ((k, (1,)), (v, (1,)), (k_scales, (2, 1)), (v_scales, (2, 1))):
            if t.stride()[3:] != last and not (t.dim() == 5 and groups == 1 and t.stride(4) == 1):
                raise ValueError("Cache: rows of codes and of scales must be contiguous")
        for a, b in ((k, v), (k_scales, v_scales)):
            if any(n > 1 and x != y for n, x, y in zip(a.shape[:3], a.stride(), b.stride())):
                raise ValueError("Cache: keys and values must have the same strides")
        device = k.get_device()
        if any(t.get_device() != device for t in (k_scales, v, v_scales)):
            raise ValueError("Cache: all tensors must be on one device")
        self.k, self.k_scales, self.v, self.v_scales = k, k_scales, v, v_scales
        self.pages, self.heads, self.page, self.head_dim, self.group, self.dtype = pages, heads, page, head_dim, group, dtype
        self._struct = _Kv4Cache(
            k.data_ptr(), v.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), pages, heads, page, head_dim, group,
            ROW_TYPES[dtype], k.stride(0), k.stride(1), k.stride(2), *(2 * n for n in k_scales.stride()[:3]))
        self._ref = ctypes.addressof(self._struct)


def empty_cache(pages: int, heads: int, page: int, head_dim: int, group: int = 64, dtype=torch.bfloat16,
                device="cuda") -> Cache:
    """A cache of ``pages`` pages of ``page`` tokens, its content undefined: rows that a call looks at
    must have been written. Groups of 32 columns are the most accurate; 64 and 128 take less room."""
    if group not in GROUPS or head_dim % group:
        raise ValueError(f"empty_cache: a scale covers 32, 64 or 128 columns, a divisor of head_dim {head_dim}; got {group}")
    parts = []
    for _ in range(2):
        parts += [torch.empty((pages, heads, page, head_dim // 2), dtype=torch.uint8, device=device),
                  torch.empty((pages, heads, page, head_dim // group, 2), dtype=dtype, device=device)]
    return Cache(*parts)


def slots(table: torch.Tensor, positions: torch.Tensor, page: int) -> torch.Tensor:
    """The slots (int64, of positions' shape [batch, n]) of each sequence's positions, through its pages table
    [batch, width]; -1 where a position is negative or past the table, or its page is."""
    column = torch.div(positions, page, rounding_mode="floor").long()
    inside = (positions >= 0) & (column < table.shape[1])
    if table.shape[1] == 0:
        return torch.full_like(column, -1)
    pages = torch.gather(table, 1, column.clamp(0, table.shape[1] - 1)).long()
    return torch.where(inside & (pages >= 0), pages * page + positions % page, -1)


def _token_rows(call: str, name: str, t: torch.Tensor, tokens: int, cache: Cache):
    """(pointer, token stride, head stride) of rows [tokens, heads, head_dim] of the cache's type."""
    if t.dtype is not cache.dtype:
        raise TypeError(f"{call}: {name} must be {cache.dtype} as the cache's scales, got {t.dtype}")
    if t.shape != (tokens, cache.heads, cache.head_dim):
        raise ValueError(f"{call}: {name} must be [{tokens}, {cache.heads}, {cache.head_dim}], got {tuple(t.shape)}")
    ld_token, ld_head, unit = t.stride()
    if unit != 1:
        raise ValueError(f"{call}: {name} must have unit column stride")
    return t.data_ptr(), ld_token, ld_head


def _slots(call: str, slots: torch.Tensor):
    if slots.dim() != 1:
        raise ValueError(f"{call}: slots must have one dimension, a slot for each token")
    wide = slots.dtype is torch.int64
    return _flat(slots, torch.int64 if wide else torch.int32, "slots"), wide, slots.shape[0]


def write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: Cache, stream=None) -> None:
    """Rows k and v [tokens, heads, head_dim] quantized into the cache's ``slots`` [tokens] (int32
    or int64; a token whose slot is outside the cache is skipped). Each slot at most once
    (bq_kv4_write)."""
    dev = _here("write", "k v slots cache", k, v, slots, cache.k)
    at, wide, tokens = _slots("write", slots)
    kp, k_token, k_head = _token_rows("write", "k", k, tokens, cache)
    vp, v_token, v_head = _token_rows("write", "v", v, tokens, cache)
    check("bq_kv4_write", load().bq_kv4_write(cache._ref, kp, k_token, k_head, vp, v_token, v_head, tokens, at, wide,
                                              _on(stream, dev)))


def read(cache: Cache, slots: torch.Tensor, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    """The rows of ``slots`` as 16-bit values into k and v [tokens, heads, head_dim]; zeros for a slot
    outside the cache (bq_kv4_read)."""
    dev = _here("read", "cache slots k v", cache.k, slots, k, v)
    at, wide, tokens = _slots("read", slots)
    kp, k_token, k_head = _token_rows("read", "k", k, tokens, cache)
    vp, v_token, v_head = _token_rows("read", "v", v, tokens, cache)
    check("bq_kv4_read", load().bq_kv4_read(cache._ref, at, wide, tokens, kp, k_token, k_head, vp, v_token, v_head,
                                            _on(stream, dev)))


def _query_shape(call: str, q: torch.Tensor, cache: Cache):
    if q.dtype is not cache.dtype:
        raise TypeError(f"{call}: q must be {cache.dtype} as the cache's scales, got {q.dtype}")
    shape = q.shape
    if len(shape) != 4 or shape[3] != cache.head_dim or shape[2] % cache.heads:
        raise ValueError(f"{call}: q must be [batch, queries, a multiple of {cache.heads} heads, {cache.head_dim}], got "
                         f"{tuple(shape)}")
    if shape[2] > 1 << 16 or shape[1] * shape[2] > 1 << 20:
        raise ValueError(f"{call}: {shape[1]} queries of {shape[2]} heads are more than a call takes")
    return shape


def empty_workspace(q: torch.Tensor, cache: Cache) -> torch.Tensor:
    """Scratch for ``attend`` calls with q's queries and heads, of any batch and any lengths: 2 to 8 MB. Calls that
    may run at the same time (other streams, graphs that are replayed together) need one each."""
    _, n_q, q_heads, dim = _query_shape("empty_workspace", q, cache)
    size = load().bq_kv4_workspace_bytes(cache.heads, dim, max(n_q, 1), max(q_heads, cache.heads))
    if size < 0:
        raise ValueError(f"empty_workspace: {n_q} queries of {q_heads} heads are more than a call takes")
    return torch.empty(max(size, 16), dtype=torch.uint8, device=q.device)


def attend(q: torch.Tensor, cache: Cache, table: torch.Tensor, lengths: torch.Tensor, out: torch.Tensor,
           workspace: torch.Tensor, scale: Optional[float] = None, window: int = 0, lse: Optional[torch.Tensor] = None,
           stream=None) -> None:
    """Attention of q [batch, queries, q_heads, head_dim], the last tokens of each sequence, over their
    cache -> out of q's shape (bq_kv4_attend).

    ``table`` int32 [batch, width]: the page of each run of cache.page positions; ``lengths`` int32
    [batch], the queries' own tokens among them, which must have been written. Query i sees the positions up to
    ``lengths - queries + i``, with ``window`` only the last ``window`` of them. Query head h reads key-value head
    ``h // (q_heads / heads)``. ``scale`` is head_dim ** -0.5 where not given. ``lse`` float32 [batch, queries,
    q_heads] takes the logarithm of each softmax's sum. A query that sees nothing gives zeros, and
    minus infinity in ``lse``. ``workspace`` is ``empty_workspace``'s."""
    dev = _here("attend", "q cache table lengths out workspace lse", q, cache.k, table, lengths, out, workspace, lse)
    batch, n_q, q_heads, dim = _query_shape("attend", q, cache)
    if out.shape != q.shape or out.dtype is not q.dtype:
        raise ValueError(f"attend: out must be {tuple(q.shape)} {q.dtype}, got {tuple(out.shape)} {out.dtype}")
    q_batch, q_query, q_head, unit = q.stride()
    o_batch, o_query, o_head, o_unit = out.stride()
    if unit != 1 or o_unit != 1:
        raise ValueError("attend: q and out must have unit column stride")
    if table.dtype is not torch.int32 or table.dim() != 2 or table.shape[0] != batch:
        raise ValueError(f"attend: table must be int32 [{batch}, width], got {table.dtype} {tuple(table.shape)}")
    width = table.shape[1]
    ld_table, t_unit = table.stride()
    if t_unit != 1 and width > 1:
        raise ValueError("attend: table must have unit column stride")
    if lengths.shape != (batch,):
        raise ValueError(f"attend: lengths must be [{batch}], got {tuple(lengths.shape)}")
    if lse is not None and lse.shape != q.shape[:3]:
        raise ValueError(f"attend: lse must be {tuple(q.shape[:3])}, got {tuple(lse.shape)}")
    if not workspace.is_contiguous():
        raise ValueError("attend: expected a contiguous workspace")
    check("bq_kv4_attend", load().bq_kv4_attend(
        cache._ref, q.data_ptr(), q_batch, q_query, q_head, batch, n_q, q_heads, table.data_ptr(), ld_table, width,
        _flat(lengths, torch.int32, "lengths"), dim ** -0.5 if scale is None else scale, window, out.data_ptr(), o_batch,
        o_query, o_head, _flat(lse, torch.float32, "lse") if lse is not None else None, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _on(stream, dev)))
