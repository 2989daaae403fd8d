"""A mixture-of-experts layer whose output is an all-reduce payload, on one GPU.

W ranks hold the experts of a layer in equal consecutive shares, as in ``topology`` W
buffers of one GPU's memory. Each rank sees every token and the router's choices, computes
its own experts' part of the output, and the parts are summed by one of the wire
topologies. Two forms of a rank's part:

* ``decode_part``: a decode step's few tokens, 4-bit expert weights, no gathered copies:
  sort -> gate and up products -> activation -> down products -> combine;
* ``part`` / ``part_grad``: any experts (a callable on rows sorted by expert), with the
  gradients with respect to the tokens and the router's weights, for prefill and training:
  sort -> gather -> experts -> combine, and back.
"""
from __future__ import annotations

from typing import Callable, List, NamedTuple, Sequence

import torch

from . import experts, topology, w4


class ExpertWeights(NamedTuple):
    """One rank's experts in 4 bits: the gate and up projections stacked, and the down
    projection, each (codes, scales) as ``w4.quant_w4`` writes them."""
    first: int              # id of this rank's first expert
    gate_up: Sequence       # codes [n_experts, 2 * inner, hidden / 2], scales
    down: Sequence          # codes [n_experts, hidden, inner / 2], scales


def quantize_experts(first: int, gate_up: torch.Tensor, down: torch.Tensor, group: int = 32) -> ExpertWeights:
    """BF16 (or FP16) expert weights [n_experts, 2 * inner, hidden] and [n_experts, hidden,
    inner] -> 4-bit weights with scales of the same type."""
    def quantized(x):
        q, s = w4.empty_w4(x.shape[1], x.shape[2], group, x.dtype, x.device, lead=x.shape[:1])
        w4.quant_w4(x, q, s)
        return q, s
    return ExpertWeights(first, quantized(gate_up), quantized(down))


def _plan(ids: torch.Tensor, first: int, n_experts: int) -> experts.Plan:
    plan = experts.empty_plan(ids.shape[0], ids.shape[1], n_experts, ids.device)
    experts.sort(ids - first if first else ids, n_experts, *plan)
    return plan


def decode_part(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w: ExpertWeights) -> torch.Tensor:
    """One rank's part of the layer's output for a few tokens x [tokens, hidden]; ids and
    weights [tokens, top_k] are the router's choice among all ranks' experts."""
    tokens, top_k = ids.shape
    n_experts, wide = w.gate_up[0].shape[:2]
    plan = _plan(ids, w.first, n_experts)
    both = torch.empty((tokens * top_k, wide), dtype=x.dtype, device=x.device)
    w4.matvec_w4_experts(x, *w.gate_up, plan.offsets, both, order=plan.order, top_k=top_k)
    gate, up = both.chunk(2, dim=1)
    act = torch.nn.functional.silu(gate) * up
    rows = torch.empty((tokens * top_k, x.shape[1]), dtype=x.dtype, device=x.device)
    w4.matvec_w4_experts(act, *w.down, plan.offsets, rows)
    out = torch.empty_like(x)
    experts.combine(rows, weights, plan.inverse, out)
    return out


def decode_layer(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, ranks: Sequence[ExpertWeights],
                 mode: str = "i8_a2a") -> List[torch.Tensor]:
    """The whole layer: every rank's part, summed through the wire mode ``mode``: a ring,
    all-to-all or all-gather mode of ``topology.MODES``, or an empty name for a sum in float32.
    Returns what the owners hold: one tensor for the all-to-all modes, row shards for the ring
    and all-gather modes. ``i8`` and ``mx`` are round trips of one tensor there, which sum
    nothing, and raise ValueError."""
    reduce = topology.select_mode(mode)
    if reduce in (topology.i8_roundtrip, topology.mx_roundtrip):
        raise ValueError(f"wire mode {mode!r} is one tensor's round trip and sums no parts; the all-gather modes that "
                         "do are 'i8_ag' and 'e4m3_ag'")
    parts = [decode_part(x, ids, weights, w) for w in ranks]
    if reduce is None:
        return [torch.stack([p.float() for p in parts]).sum(0).to(x.dtype)]
    owned = reduce(parts)[2]
    return [owned] if isinstance(owned, torch.Tensor) else list(owned)


class Part(NamedTuple):
    """A rank's part and what its backward pass needs."""
    out: torch.Tensor
    plan: experts.Plan
    rows_in: torch.Tensor
    rows_out: torch.Tensor


def part(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, first: int, n_experts: int,
         forward: Callable) -> Part:
    """``forward(rows, offsets)`` maps rows [tokens * top_k, hidden], sorted by expert (zeros
    past offsets[-1]), to as many output rows."""
    plan = _plan(ids, first, n_experts)
    rows = torch.empty((ids.numel(), x.shape[1]), dtype=x.dtype, device=x.device)
    experts.gather(x, plan.inverse, plan.offsets, rows)
    y = forward(rows, plan.offsets)
    out = torch.empty((x.shape[0], y.shape[1]), dtype=y.dtype, device=x.device)
    experts.combine(y, weights, plan.inverse, out)
    return Part(out, plan, rows, y)


def part_grad(dout: torch.Tensor, weights: torch.Tensor, p: Part, backward: Callable):
    """(dx, dweights) for the gradient dout of ``part``'s output; ``backward(drows_out, rows_in,
    offsets)`` gives the gradient with respect to the experts' input rows."""
    drows = torch.empty_like(p.rows_out)
    dweights = torch.empty_like(weights)
    experts.combine_grad(dout, p.rows_out, weights, p.plan.inverse, p.plan.offsets, drows, dweights)
    drows_in = backward(drows, p.rows_in, p.plan.offsets)
    dx = torch.empty((dout.shape[0], drows_in.shape[1]), dtype=drows_in.dtype, device=dout.device)
    experts.gather_grad(drows_in, p.plan.inverse, dx)
    return dx, dweights
