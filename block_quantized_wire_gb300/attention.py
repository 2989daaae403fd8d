"""A decode step of an attention layer whose output is an all-reduce payload, on one GPU.

W ranks hold the heads of a layer in shares, as in ``topology`` W buffers of one GPU's memory, and
each its own pages of the heads' cache. Each rank sees every token: its 4-bit projection gives
queries, keys and values of its heads, keys and values go into its 4-bit cache, the queries attend over
it, and the 4-bit output projection gives the rank's part. The parts are summed by one of the wire
topologies, as ``moe.decode_layer`` sums the expert layer's.
"""
from __future__ import annotations

from typing import Callable, List, NamedTuple, Optional, Sequence

import torch

from . import kv4, moe, w4


class HeadWeights(NamedTuple):
    """One rank's heads in 4 bits: the projections of queries, keys and values stacked, and the output
    projection, each (codes, scales) as ``w4.quant_w4`` writes them."""
    q_heads: int
    heads: int       # key-value heads
    qkv: Sequence    # codes [(q_heads + 2 * heads) * head_dim, hidden / 2], scales
    out: Sequence    # codes [hidden, q_heads * head_dim / 2], scales


def quantize_heads(q_heads: int, heads: int, qkv: torch.Tensor, out: torch.Tensor, group: int = 32) -> HeadWeights:
    """BF16 (or FP16) weights [(q_heads + 2 * heads) * head_dim, hidden] and [hidden, q_heads *
    head_dim] -> 4-bit weights with scales of the same type."""
    def quantized(x):
        q, s = w4.empty_w4(x.shape[0], x.shape[1], group, x.dtype, x.device)
        w4.quant_w4(x, q, s)
        return q, s
    return HeadWeights(q_heads, heads, quantized(qkv), quantized(out))


def decode_part(x: torch.Tensor, w: HeadWeights, cache: kv4.Cache, table: torch.Tensor, lengths: torch.Tensor,
                queries: int = 1, rotate: Optional[Callable] = None, workspace: Optional[torch.Tensor] = None,
                window: int = 0) -> torch.Tensor:
    """One rank's part of the layer's output for x [batch * queries, hidden], the last ``queries`` tokens of
    each sequence; ``table`` and ``lengths`` as ``kv4.attend`` takes them, these tokens counted. A
    sequence whose length is 0 (a padded request) writes nothing and gives zeros. Lengths stay on the device and are not checked:
    give a sequence its pages before it needs them. Of one longer than its table (``table.shape[1] * cache.page``) the tokens past
    the table are not written, and its queries see what queries of a sequence that just fills the table see; other sequences are
    as always.
    ``rotate(q, k, positions)`` maps queries [batch, queries, q_heads, head_dim] and keys [batch, queries, heads, head_dim]
    at positions [batch, queries] to what is attended with and cached."""
    batch, dim = lengths.shape[0], cache.head_dim
    both = torch.empty((x.shape[0], w.qkv[0].shape[0]), dtype=x.dtype, device=x.device)
    w4.matvec_w4(x, *w.qkv, both)
    q, k, v = both.view(batch, queries, w.q_heads + 2 * w.heads, dim).split([w.q_heads, w.heads, w.heads], dim=2)
    positions = lengths[:, None] - queries + torch.arange(queries, dtype=torch.int32, device=x.device)
    if rotate is not None:
        q, k = rotate(q, k, positions)
    slots = kv4.slots(table, positions, cache.page)
    kv4.write(k.flatten(0, 1), v.flatten(0, 1), slots.flatten(), cache)
    heads = torch.empty((batch, queries, w.q_heads, dim), dtype=x.dtype, device=x.device)
    if workspace is None:
        workspace = kv4.empty_workspace(q, cache)
    kv4.attend(q, cache, table, lengths, heads, workspace, window=window)
    out = torch.empty_like(x)
    w4.matvec_w4(heads.view(x.shape[0], w.q_heads * dim), *w.out, out)
    return out


def decode_layer(x: torch.Tensor, ranks: Sequence[HeadWeights], caches: Sequence[kv4.Cache], table: torch.Tensor,
                 lengths: torch.Tensor, mode: str = "i8_a2a", queries: int = 1, rotate: Optional[Callable] = None,
                 window: int = 0) -> List[torch.Tensor]:
    """The whole layer: every rank's part, summed through the wire mode ``mode`` and returned as
    ``moe.decode_layer`` does. Each rank has a cache of its own; all go by the same table."""
    reduce = moe.reduction(mode)
    if len(ranks) != len(caches):
        raise ValueError(f"decode_layer: {len(ranks)} ranks need a cache each, got {len(caches)} caches")
    parts = [decode_part(x, w, cache, table, lengths, queries, rotate, window=window) for w, cache in zip(ranks, caches)]
    return moe.summed(parts, reduce)
