"""The expert layer's composition without a GPU: which wire modes sum its parts."""
import pytest

from block_quantized_wire_gb300 import moe, topology


@pytest.mark.parametrize("mode", ["i8", "mx", " I8\t", "Mx"])
def test_a_round_trip_of_one_tensor_is_refused_before_any_work(mode):
    assert topology.select_mode(mode) in (topology.i8_roundtrip, topology.mx_roundtrip)
    with pytest.raises(ValueError, match="one tensor's round trip.*'i8_ag'"):
        moe.decode_layer(None, None, None, [None], mode)


@pytest.mark.parametrize("mode", ["i8-ring", "int8"])
def test_an_unknown_mode_is_refused_before_any_work(mode):
    with pytest.raises(ValueError, match="unknown wire mode"):
        moe.decode_layer(None, None, None, [None], mode)


@pytest.mark.parametrize("mode", sorted(set(topology.MODES) - {"i8", "mx"}) + ["", None])
def test_every_other_mode_sums_the_parts(mode, monkeypatch):
    import torch
    parts = [torch.full((4, 128), float(r)) for r in range(2)]
    monkeypatch.setattr(moe, "decode_part", lambda x, ids, weights, w: parts[w])
    seen = []

    def fake(xs, stream=None):
        seen.append(xs)
        return None, None, xs[0] + xs[1]
    monkeypatch.setattr(topology, "MODES", {m: fake for m in topology.MODES})
    (out,) = moe.decode_layer(parts[0], None, None, [0, 1], mode)
    assert torch.equal(out, parts[0] + parts[1]) and len(seen) == (1 if mode else 0)


def test_a_ring_of_one_rank_materializes_its_owner():
    # one rank: no hop runs, so the owner's copy comes from its own payload
    import torch

    def empty(n, device):
        return None, torch.zeros(n), torch.zeros(1)

    def quant(x, q, s, stream):
        q.copy_(x.reshape(-1) * 2)

    def dequant(q, s, out, stream):
        out.copy_((q / 2).view(out.shape))

    wire = topology.Wire(empty, quant, dequant, None, None)
    x = torch.arange(256.0).view(2, 128)
    outs, finals, owners = topology.ring(wire, [x])
    assert torch.equal(outs[0], x) and torch.equal(finals[0][0], 2 * x.reshape(-1))
    assert torch.equal(owners[0], x)
