"""Attention over the 4-bit cache where its work is cut and joined differently, over strides of every order, at the ends of the
number ranges, and with workspaces that calls share. Reference and bounds are those of test_gpu_kv4."""
import numpy as np
import pytest
import torch

from block_quantized_wire_gb300 import kv4
from tests.test_gpu_kv4 import (TYPES, check, fill, guarded_cache, quantized, reference, run, same_bits, table_of)

pytestmark = pytest.mark.gpu


def problem(seed, lens, n_q, q_heads, heads, dim, group, page, dtype=torch.bfloat16, cache=None):
    rng = np.random.default_rng(seed)
    width, pages = -(-max(max(lens), 1) // page) + 1, sum(-(-n // page) for n in lens) + 2
    if cache is None:
        cache = kv4.empty_cache(pages, heads, page, dim, group, dtype)
    fill(rng, cache)
    table = table_of(rng, lens, page, width, pages)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.from_numpy(rng.standard_normal((len(lens), n_q, q_heads, dim)).astype(np.float32)).to(dtype).cuda()
    return q, cache, table, lengths


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("group", [32, 64, 128])
def test_rows_with_offsets_of_any_size_beside_their_range(name, group):
    # means of 0 to 1000 ranges, around 32 steps too; ranges down to the smallest values of the type
    dtype = TYPES[name][0]
    torch.manual_seed(group)
    x = torch.randn(2048, 2, 128, device="cuda")
    x = x + torch.randn(2048, 2, 1, device="cuda").sign() * torch.logspace(-1, 3, 2048, device="cuda")[:, None, None]
    x = (x * torch.logspace(-7, 1, 8, device="cuda").repeat(256)[:, None, None]).to(dtype)
    cache = kv4.empty_cache(32, 2, 64, 128, group, dtype)
    kv4.write(x, -x, torch.arange(2048, device="cuda"), cache)
    for rows, codes, pairs in ((x, cache.k, cache.k_scales), (-x, cache.v, cache.v_scales)):
        want, want_pairs, _ = quantized(rows, group)
        assert np.array_equal(codes.transpose(1, 2).reshape(2048, 2, 64).cpu().numpy(), want)
        assert torch.equal(pairs.transpose(1, 2).reshape(want_pairs.shape).cpu(), want_pairs)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 160, 161])
@pytest.mark.parametrize("page", [32, 40, 96])
def test_lengths_around_a_tile(n, page):
    q, cache, table, lengths = problem(n, [n, n - 1, n + 1], 1, 4, 2, 64, 64, page)
    check(*run(q, cache, table, lengths), reference(q, cache, table, lengths, 0.125, 0, 8))


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 64, 100])
@pytest.mark.parametrize("page", [16, 32, 50, 64])
def test_windows_around_a_tile(window, page):
    q, cache, table, lengths = problem(window, [97, 128, 200, 5], 3, 4, 2, 128, 32, page, torch.float16)
    check(*run(q, cache, table, lengths, window=window), reference(q, cache, table, lengths, 128 ** -0.5, window, 11))


@pytest.mark.parametrize("shape", [([40] * 300 + [0, 1, 700], 1, 4, 4, 64, 64, 64), ([9, 0] * 400, 1, 2, 2, 64, 32, 16),
                                   ([70] * 100, 1, 32, 8, 64, 64, 48)])
def test_more_items_than_the_workspace_has_words(shape):
    lens, *rest = shape
    q, cache, table, lengths = problem(len(lens), lens, *rest)
    out, lse = run(q, cache, table, lengths)
    check(out, lse, reference(q, cache, table, lengths, 0.125, 0, 8))


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("shape", [([20000], 1, 1, 1, 64, 32, 64), ([12000, 3], 1, 20, 2, 128, 128, 32), ([9000, 100], 2, 3, 1, 192, 64, 24),
                                   ([8000], 2, 8, 1, 256, 32, 128), ([6000, 0, 6000], 12, 3, 1, 64, 64, 128)])
def test_sequences_on_many_shares(shape, name):
    lens, *rest = shape
    q, cache, table, lengths = problem(sum(lens), lens, *rest, dtype=TYPES[name][0])
    check(*run(q, cache, table, lengths), reference(q, cache, table, lengths, rest[3] ** -0.5, 0, TYPES[name][1]))


@pytest.mark.parametrize("dim,group", [(64, 32), (128, 64), (192, 32), (256, 128)])
@pytest.mark.parametrize("page", [64, 20])
def test_tokens_before_heads(dim, group, page):
    lens = [300, 64, 7]
    cache, guards = guarded_cache(sum(-(-n // page) for n in lens) + 2, 3, page, dim, group, torch.bfloat16, True)
    q, cache, table, lengths = problem(dim, lens, 2, 9, 3, dim, group, page, cache=cache)
    check(*run(q, cache, table, lengths), reference(q, cache, table, lengths, dim ** -0.5, 0, 8))
    assert all(g.bands_intact() for g in guards)


def test_queries_and_outputs_of_other_strides():
    # heads before batches in memory, and one row for all queries
    q, cache, table, lengths = problem(3, [77, 300], 4, 6, 2, 128, 64, 32)
    want, want_lse = run(q, cache, table, lengths)
    turned = q.permute(2, 1, 0, 3).contiguous().permute(2, 1, 0, 3)
    out = torch.empty(6, 2, 4, 128, dtype=q.dtype, device="cuda").permute(1, 2, 0, 3)
    ws = kv4.empty_workspace(q, cache)
    kv4.attend(turned, cache, table, lengths, out, ws)
    assert same_bits(out, want)
    same = q[:, :1].expand(2, 4, 6, 128)
    check(*run(same, cache, table, lengths), reference(same, cache, table, lengths, 128 ** -0.5, 0, 8))


@pytest.mark.parametrize("up", [-70, -40, 40, 60])
def test_scales_of_any_size(up):
    # keys, queries and values times powers of two that cancel in the scores; sums of p z stay finite
    q, cache, table, lengths = problem(5, [500, 33], 1, 4, 1, 128, 64, 32)
    cache.k_scales *= 2.0 ** up
    cache.v_scales *= 2.0 ** up
    q = torch.ldexp(q.float(), torch.tensor(-up, device="cuda")).to(q.dtype)
    out, lse = run(q, cache, table, lengths)
    o, l, bound, bound_lse = reference(q, cache, table, lengths, 128 ** -0.5, 0, 8)
    bound -= 2.0 ** -25 - 2.0 ** (up - 25)  # the bound's last term is for values of about 1
    check(out, lse, (o, l, bound, bound_lse))


def test_constant_and_zero_values():
    # scales of 0 (constant rows) beside large offsets, and values that are all zero
    q, cache, table, lengths = problem(6, [300, 40, 1], 1, 8, 2, 64, 32, 16)
    cache.v_scales[..., 0] = 0
    cache.v_scales[..., 1] *= 1e30
    out, lse = run(q, cache, table, lengths)
    o = out.double().cpu().numpy()
    want = reference(q, cache, table, lengths, 0.125, 0, 8)
    assert np.all(np.abs(o - want[0]) <= 1e30 * 2.0 ** -10 + 2.0 ** -8 * np.abs(want[0]))  # 300 / 16 + 64 steps of 2^-23, one rounding
    cache.v_scales.zero_()
    out, lse2 = run(q, cache, table, lengths)
    check(out, lse2, reference(q, cache, table, lengths, 0.125, 0, 8))
    assert not out.any()
    q.zero_()
    cache.v_scales[..., 0], cache.v_scales[..., 1] = 0.25, 1.0
    check(*run(q, cache, table, lengths), reference(q, cache, table, lengths, 0.125, 0, 8))


def test_not_a_number_stays_in_its_rows():
    # a NaN key reaches every column of the queries that see it, a NaN group of values its columns only
    q, cache, table, lengths = problem(7, [200, 200], 1, 4, 2, 128, 64, 32)
    clean, _ = run(q, cache, table, lengths)
    page = int(table[0, 2])
    cache.v_scales[page, 1, 3, 0] = float("nan")
    out, _ = run(q, cache, table, lengths)
    bad = torch.isnan(out.float())
    assert bool(bad[0, :, 2:, :64].all()) and int(bad.sum()) == 2 * 64 and same_bits(out[~bad], clean[~bad])
    cache.k_scales[page, 0, 5, 1, 0] = float("nan")
    out, lse = run(q, cache, table, lengths)
    assert bool(torch.isnan(out[0, :, :2].float()).all()) and bool(torch.isnan(lse[0, :, :2]).all())
    assert same_bits(out[1], clean[1])
    q[1, 0, 3, 7] = float("nan")
    out, _ = run(q, cache, table, lengths)
    assert bool(torch.isnan(out[1, 0, 3].float()).all()) and same_bits(out[1, 0, :3], clean[1, 0, :3])


def test_graphs_that_share_a_workspace():
    # of different lengths, replayed in turn on one stream
    parts, ws, graphs, outs, wants = [], None, [], [], []
    for seed, lens in ((8, [3000, 20]), (9, [10, 1000]), (10, [0, 64])):
        q, cache, table, lengths = problem(seed, lens, 1, 8, 2, 128, 64, 64)
        ws = kv4.empty_workspace(q, cache) if ws is None else ws
        wants.append(run(q, cache, table, lengths)[0])
        out = torch.empty_like(q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kv4.attend(q, cache, table, lengths, out, ws)
        parts.append((q, cache, table, lengths))
        graphs.append(graph)
        outs.append(out)
    for i in (0, 1, 2, 0, 2, 1, 0):
        outs[i].fill_(float("nan"))
        graphs[i].replay()
        torch.cuda.synchronize()
        assert same_bits(outs[i], wants[i])


def test_a_write_and_an_attention_right_after_another():
    # attention sees what the write before it on the stream wrote, a hundred steps on end
    torch.manual_seed(0)
    cache = kv4.empty_cache(8, 2, 16, 64, 32)
    for c in (cache.k, cache.v):
        c.zero_()
    for s in (cache.k_scales, cache.v_scales):
        s.zero_()
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    rows = torch.randn(100, 2, 64, device="cuda").to(torch.bfloat16)
    q = torch.randn(1, 1, 4, 64, device="cuda").to(torch.bfloat16)
    ws, outs = kv4.empty_workspace(q, cache), torch.empty(100, 1, 1, 4, 64, dtype=q.dtype, device="cuda")
    lengths = torch.arange(1, 101, dtype=torch.int32, device="cuda")
    slots = torch.arange(100, device="cuda")
    torch.cuda.synchronize()
    for i in range(100):
        kv4.write(rows[i:i + 1], rows[i:i + 1], slots[i:i + 1], cache)
        kv4.attend(q, cache, table, lengths[i:i + 1], outs[i], ws)
    for i in (0, 1, 31, 32, 50, 99):
        check(outs[i], None, reference(q, cache, table, lengths[i:i + 1], 0.125, 0, 8))
