"""The attention layer's forms that a server meets: no requests, several tokens a request, a window, FP16, an own workspace,
sequences that fill their table, every kind of wire mode. The layer of test_gpu_kv4 is what is compared with."""
import pytest
import torch

from block_quantized_wire_gb300 import attention, kv4, topology, w4
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


def by_hand(x, rank, cache, table, lengths, queries, window):
    """A part's operators one after another, the slots of the tokens found position by position."""
    batch, dim = len(lengths), cache.head_dim
    both = torch.empty(x.shape[0], rank.qkv[0].shape[0], dtype=x.dtype, device="cuda")
    w4.matvec_w4(x, *rank.qkv, both)
    nq, nk = rank.q_heads * dim, rank.heads * dim
    q, k, v = (both[:, a:b].contiguous() for a, b in ((0, nq), (nq, nq + nk), (nq + nk, nq + 2 * nk)))
    at = []
    for b, n in enumerate(lengths.tolist()):
        for j in range(n - queries, n):
            at.append(int(table[b, j // cache.page]) * cache.page + j % cache.page if j >= 0 else -1)
    kv4.write(k.view(-1, rank.heads, dim), v.view(-1, rank.heads, dim), torch.tensor(at, device="cuda"), cache)
    q = q.view(batch, queries, rank.q_heads, dim)
    heads, out = torch.empty_like(q), torch.empty_like(x)
    kv4.attend(q, cache, table, lengths, heads, kv4.empty_workspace(q, cache), window=window)
    w4.matvec_w4(heads.view(x.shape[0], nq), *rank.out, out)
    return out


@pytest.mark.parametrize("queries,window", [(1, 0), (1, 7), (4, 0), (5, 12)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_part_is_its_operators_one_after_another(dtype, queries, window):
    torch.manual_seed(queries + window)
    hidden, q_heads, heads, dim, page, lens = 256, 6, 2, 128, 16, [70, 3, 0, 33, 16]
    qkv = (torch.randn((q_heads + 2 * heads) * dim, hidden, device="cuda") / 16).to(dtype)
    o = (torch.randn(hidden, q_heads * dim, device="cuda") / 28).to(dtype)
    rank = attention.quantize_heads(q_heads, heads, qkv, o)
    a, b = (kv4.empty_cache(30, heads, page, dim, 64, dtype) for _ in range(2))
    rows = torch.randn(480, heads, dim, device="cuda").to(dtype)
    for c in (a, b):
        for t in (c.k, c.v, c.k_scales, c.v_scales):
            t.zero_()
        kv4.write(rows, rows * 0.5, torch.arange(480, device="cuda"), c)
    table = torch.randperm(30, device="cuda")[:25].int().view(5, 5)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = kv4.empty_workspace(torch.empty(5, queries, q_heads, dim, dtype=dtype, device="cuda"), a)
    for step in range(2):
        x = torch.randn(5 * queries, hidden, device="cuda").to(dtype)
        got = attention.decode_part(x, rank, a, table, lengths, queries, workspace=ws, window=window)
        want = by_hand(x, rank, b, table, lengths, queries, window)
        assert torch.equal(got, want) and bool(torch.isfinite(got.float()).all())
        assert not got.view(5, queries, hidden)[2].any()  # the padded request
        for s, t in zip((a.k, a.v, a.k_scales, a.v_scales), (b.k, b.v, b.k_scales, b.v_scales)):
            assert torch.equal(s, t)
        lengths = torch.where(lengths > 0, lengths + queries, 0).int()


@pytest.mark.parametrize("mode", ["i8_ag", "e4m3_ag", "mx_ring", "mx_a2a"])
def test_a_layer_sums_its_parts_as_the_wire_mode_does(mode):
    ranks, caches, table, lengths, (x,) = a_layer(mode, steps=1)
    lengths += 1
    parts = [attention.decode_part(x, r, c, table, lengths) for r, c in zip(ranks, caches)]
    want = topology.MODES[mode](parts)[2]
    got = attention.decode_layer(x, ranks, caches, table, lengths, mode)  # writes the same rows once more
    want = [want] if isinstance(want, torch.Tensor) else list(want)
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_captured_layer_follows_its_inputs():
    ranks, caches, table, lengths, xs = a_layer("", steps=3)
    again = [kv4.Cache(*(t.clone() for t in (c.k, c.k_scales, c.v, c.v_scales))) for c in caches]
    x, lens, tab = xs[0].clone(), lengths.clone(), table.clone()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        attention.decode_layer(x, ranks, again, tab, torch.zeros_like(lens), "i8_a2a")  # writes nothing
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, = attention.decode_layer(x, ranks, again, tab, lens, "i8_a2a")
    for step, new in enumerate(xs):
        lengths += 1
        if step == 2:
            lengths[1] = 0  # a request that has ended
            table[3] = table[3].roll(1)
        want, = attention.decode_layer(new, ranks, caches, table, lengths, "i8_a2a")
        x.copy_(new), lens.copy_(lengths), tab.copy_(table)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        for a, b in zip(caches, again):
            assert torch.equal(a.k, b.k) and torch.equal(a.v_scales, b.v_scales)
