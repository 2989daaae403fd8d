"""The attention layer's forms that a server meets: no requests, several tokens a request, a window, FP16, an own workspace,
sequences that fill their table, every kind of wire mode. The layer of test_gpu_kv4 is what is compared with."""
import pytest
import torch

from block_quantized_wire_gb300 import attention, kv4, w4
from tests.test_gpu_kv4 import a_layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", ["", "i8_a2a", "mx_ring", "i8_ag"])
@pytest.mark.parametrize("queries", [1, 3])
def test_a_step_of_no_requests(mode, queries):
    ranks, caches, table, lengths, (x,) = a_layer(mode, steps=1)
    before = [t.clone() for c in caches for t in (c.k, c.v)]
    outs = attention.decode_layer(x[:0], ranks, caches, table[:0], lengths[:0], mode, queries=queries)
    assert all(o.numel() == 0 and o.dtype is x.dtype for o in outs)
    assert all(torch.equal(a, b) for a, b in zip(before, [t for c in caches for t in (c.k, c.v)]))


@pytest.mark.parametrize("queries", [1, 2])
def test_a_sequence_past_its_table_writes_nothing_and_sees_what_is_held(queries):
    # two pages of 16 a sequence: the first is full, the second has room for its last token only, the third is within its table
    (rank,), (cache,), table, lengths, (x,) = a_layer("", n_ranks=1, steps=1)
    x, table = x.repeat_interleave(queries, 0), table[:, :2].contiguous()
    full, over = (torch.tensor([a, b, 20, 0], dtype=torch.int32, device="cuda") for a, b in ((32, 32), (40, 33)))
    before = [t.clone() for t in (cache.k, cache.v)]
    got = attention.decode_part(x, rank, cache, table, over, queries)
    written = [(c != b).any(-1).any(1) for c, b in zip((cache.k, cache.v), before)]  # [pages, page]
    slots = kv4.slots(table, over[:, None] - queries + torch.arange(queries, device="cuda"), 16)
    assert slots[0].tolist() == [-1] * queries and int(slots[1, -1]) == -1
    allowed = torch.zeros_like(written[0]).view(-1)
    allowed[slots[slots >= 0]] = True
    assert all(bool((w.view(-1) == allowed).all()) for w in written)
    held = [t.clone() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)]
    want = attention.decode_part(x, rank, cache, table, full, queries)  # writes what the first two did not: put back
    for t, h in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), held):
        t.copy_(h)
    q = torch.empty(4, queries, 4, 64, dtype=x.dtype, device="cuda")
    both = torch.empty(4 * queries, 8 * 64, dtype=x.dtype, device="cuda")
    w4.matvec_w4(x, *rank.qkv, both)
    q.copy_(both.view(4, queries, 8, 64)[:, :, :4])
    heads, ws = torch.empty_like(q), kv4.empty_workspace(q, cache)
    kv4.attend(q, cache, table, full, heads, ws)
    out = torch.empty_like(x)
    w4.matvec_w4(heads.view(4 * queries, 256), *rank.out, out)
    assert torch.equal(got, out) and torch.equal(got[2 * queries:], want[2 * queries:])
