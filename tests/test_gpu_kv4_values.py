"""Attention over the 4-bit cache by checks that see a single lost position, and over values of every size."""
import math

import numpy as np
import pytest
import torch

from block_quantized_wire_gb300 import _lib, build, codec, kv4
from tests.kv4_checks import BITS, check_rows, check_shares, marked_codes, rows_of, shares
from tests.test_gpu_kv4 import TYPES, fill, run, table_of
from tests.test_gpu_kv4_ranges import problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("shape", [([9000, 100], 1, 8, 1, 64, 32, 64), ([2049, 1, 700], 1, 8, 4, 128, 64, 32), ([3000], 4, 16, 2, 128, 128, 100),
                                   ([40, 33, 0, 500], 2, 15, 3, 192, 64, 24), ([1500], 1, 4, 2, 256, 32, 16), ([70] * 60, 1, 4, 4, 64, 64, 10)])
def test_rows_are_as_accurate_as_their_roundings(shape, name):
    lens, *rest = shape
    q, cache, table, lengths = problem(sum(lens), lens, *rest, dtype=TYPES[name][0])
    out, lse = run(q, cache, table, lengths)
    check_rows(out, lse, rows_of(q, cache, table, lengths, rest[3] ** -0.5), BITS[name])


# lengths, queries, q heads, heads, dim, group, page, window: one and many CTAs a sequence, shares that begin within sequences, one-tile
# items, more items than words, 8 and 16 rows, several chunks of rows
SHARES = [([65000], 1, 1, 1, 64, 64, 64, 0), ([20000], 1, 8, 1, 64, 32, 64, 0), ([20000, 0, 33], 1, 9, 1, 128, 64, 32, 0),
          ([5000, 9000, 1, 31, 32, 64, 0, 2], 1, 8, 2, 128, 32, 100, 0), ([700] * 70, 1, 8, 8, 64, 64, 16, 0),
          ([65] * 600, 1, 2, 2, 64, 32, 24, 0), ([20] * 200, 8, 16, 4, 64, 64, 32, 0), ([6000, 90], 40, 4, 1, 128, 128, 64, 0),
          ([3000, 200], 3, 12, 2, 192, 32, 10, 0), ([4000], 1, 8, 1, 256, 128, 128, 0), ([9000, 50], 1, 4, 1, 64, 64, 64, 1000),
          ([900, 2, 400], 5, 4, 2, 256, 64, 48, 33), ([128 * 37] * 5, 1, 8, 4, 128, 64, 128, 0)]


@pytest.mark.parametrize("shape", SHARES)
def test_every_position_counts_once(shape):
    # scores of zero and values that mark their position: a position lost or counted twice, anywhere, moves a column
    lens, n_q, q_heads, heads, dim, group, page, window = shape
    rng = np.random.default_rng(sum(lens))
    pages = sum(-(-n // page) for n in lens) + 2
    cache = kv4.empty_cache(pages, heads, page, dim, group, torch.float16)
    fill(rng, cache)
    table = table_of(rng, lens, page, -(-max(lens) // page) + 1, pages)
    cache.v.zero_()
    cache.v_scales[..., 0], cache.v_scales[..., 1] = 1.0, 0.0
    codes = torch.from_numpy(marked_codes(max(lens), dim)).cuda()
    packed = ((codes[:, 0::2] & 15) | ((codes[:, 1::2] & 15) << 4)).to(torch.uint8)
    for b, n in enumerate(lens):
        at = kv4.slots(table[b:b + 1], torch.arange(n, device="cuda")[None], page)[0]
        cache.v[at // page, :, at % page] = packed[:n, None]
    q = torch.zeros(len(lens), n_q, q_heads, dim, dtype=torch.float16, device="cuda")
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = run(q, cache, table, lengths, window=window)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, n in enumerate(lens):
        want = shares(n, n_q, window, dim)
        for h in range(q_heads):
            check_shares(out[b, :, h], want)
        for i in range(n_q):
            count = max(0, min(n - n_q + i + 1, window or n))
            assert np.all(np.abs(lse[b, i] - math.log(count)) <= 2.0 ** -20 * (1 + math.log(count))) if count else \
                np.all(np.isneginf(lse[b, i]))


# ---------------------------------------------------------------- values of every size
@pytest.mark.parametrize("up", [-70, -40, 0, 40, 60, 95, 97, 111, 112, 116, 120])
def test_rows_of_scales_of_any_size(up):
    # the values' scales and offsets times a power of two, which the output follows
    q, cache, table, lengths = problem(5, [900, 33], 1, 4, 1, 128, 64, 32)
    cache.v_scales *= 2.0 ** up
    check_rows(*run(q, cache, table, lengths), rows_of(q, cache, table, lengths, 128 ** -0.5), 8)
    cache.v_scales[..., 1] = 0  # without offsets, and with nothing else
    check_rows(*run(q, cache, table, lengths), rows_of(q, cache, table, lengths, 128 ** -0.5), 8)
    cache.v_scales[..., 1], cache.v_scales[..., 0] = 2.0 ** up, 0
    check_rows(*run(q, cache, table, lengths), rows_of(q, cache, table, lengths, 128 ** -0.5), 8)


def winner_of(n, winner, below, q_heads=4, n_q=1, dtype=torch.bfloat16, dim=64):
    """A sequence whose position `winner` has a score of `below` ln 2 above all others, for every query; values of about 1."""
    cache = kv4.empty_cache(-(-n // 32), 1, 32, dim, 32, dtype)
    fill(np.random.default_rng(n), cache)
    cache.k.zero_()
    cache.k_scales[..., 0], cache.k_scales[..., 1] = 1.0, 0.0
    cache.k[winner // 32, 0, winner % 32, 0] = 7
    table = torch.arange(-(-n // 32), dtype=torch.int32, device="cuda")[None]
    q = torch.zeros(1, n_q, q_heads, dim, dtype=dtype, device="cuda")
    q[..., 0] = 1
    return q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), below * math.log(2) / 7


@pytest.mark.parametrize("up", [60, 97, 112, 120, 124])
@pytest.mark.parametrize("n,below", [(40000, 15), (500, 16), (300, 8), (130000, 17)])
def test_many_small_weights_beside_a_large_one(n, below, up):
    # their sum is what counts in lse and in the output, whatever the values' size
    q, cache, table, lengths, scale = winner_of(n, n // 3, below)
    cache.v_scales[..., 0], cache.v_scales[..., 1] = 2.0 ** up, 0.0
    cache.v.fill_(0x33)  # values of 3 scales, the winner's of 1
    cache.v[n // 3 // 32, 0, n // 3 % 32] = 0x11
    out, lse = run(q, cache, table, lengths, scale=scale)
    all_of = 2.0 ** below + n - 1
    steps = (n / 16 + 64) * 2.0 ** -23
    # scores: one product, a rounding each of scale, of its product with log2 e and with x, ex2 and log: 8 steps of 2^-23 of 17 ln 2
    assert bool(((lse.double() - math.log(all_of)).abs() <= 8 * 17 * 2.0 ** -23 + steps + 2.0 ** -21).all())
    want = (2.0 ** below + 3 * (n - 1)) / all_of
    # the output's rounding, the weights' to FP16, sums of code + 8 less 8 times the weights; the scores' error above
    assert bool(((out.double() * 2.0 ** -up - want).abs() <= want * (2.0 ** -8 + 2.0 ** -11 + 16 * 17 * 2.0 ** -23) + 19 * steps).all())


# products of a weight and a scale are rounded at a power of two of the row's own: to 2^-33 of the row's largest
@pytest.mark.parametrize("name,up", [("bf16", 40), ("bf16", 100), ("f16", 23)])
@pytest.mark.parametrize("n_q,window", [(3, 0), (3, 40), (16, 70)])
def test_large_values_that_a_query_does_not_see_are_nothing_to_it(name, up, n_q, window):
    # the last position, which the last query alone sees, and with a window the first one of the first query
    dtype = TYPES[name][0]
    q, cache, table, lengths = problem(up + n_q, [200, 77, 130], n_q, 4, 2, 128, 32, 32, dtype)
    if name == "f16":
        cache.v_scales *= 2.0 ** -10
    clean, clean_lse = run(q, cache, table, lengths, window=window)
    for b, n in enumerate(lengths.tolist()):
        for j in ([n - 1, n - n_q + 1 - window] if window else [n - 1]):
            if j >= 0:
                cache.v_scales[table[b, j // 32], :, j % 32] *= 2.0 ** up
    out, lse = run(q, cache, table, lengths, window=window)
    scale = 128 ** -0.5
    check_rows(out, lse, rows_of(q, cache, table, lengths, scale, window), BITS[name])
    between = slice(1 if window else 0, n_q - 1)
    rows = [r for r in rows_of(q, cache, table, lengths, scale, window) if between.start <= r[0][1] < between.stop]
    check_rows(clean, clean_lse, rows, BITS[name])


@pytest.mark.parametrize("name,up", [("bf16", 30), ("bf16", 50), ("bf16", 90), ("f16", 23)])
@pytest.mark.parametrize("n", [33, 500, 5000])
def test_large_values_of_no_weight(name, up, n):
    # a position 2^up times larger than all others whose weight is 2^-(up + 20) of theirs
    dtype = TYPES[name][0]
    q, cache, table, lengths, scale = winner_of(n, n // 2, up + 20, dtype=dtype)
    if name == "f16":
        cache.v_scales *= 2.0 ** -10
    cache.v_scales[n // 2 // 32, 0, n // 2 % 32] *= 2.0 ** up
    out, lse = run(q, cache, table, lengths, scale=-scale)
    check_rows(out, lse, rows_of(q, cache, table, lengths, -scale), BITS[name])


@pytest.mark.parametrize("name", list(TYPES))
def test_large_weights_of_small_values(name):
    # a sink: one position takes nearly all weight and holds next to nothing, the others' part is the output
    q, cache, table, lengths, scale = winner_of(3000, 0, 12, dtype=TYPES[name][0])
    cache.v_scales[0, 0, 0] *= 2.0 ** -13
    check_rows(*run(q, cache, table, lengths, scale=scale), rows_of(q, cache, table, lengths, scale), BITS[name])


def test_offsets_of_any_size_beside_no_steps():
    # scales of 0, scores of 0: the mean of the offsets, binary32 sums and one rounding
    q, cache, table, lengths = problem(6, [300, 40, 1], 1, 8, 2, 64, 32, 16)
    q.zero_()
    cache.v_scales[..., 0] = 0
    for up in (0, 100, 20):
        cache.v_scales[..., 1] *= 2.0 ** up  # 1, 2^100, 2^120
        out = run(q, cache, table, lengths)[0].double().cpu().numpy()
        for at, want, _, w, _, _, z in rows_of(q, cache, table, lengths, 0.125):
            assert np.all(np.abs(out[at] - want) <= 2.0 ** -8 * np.abs(want) + (len(w) / 16 + 64) * 2.0 ** -23 * (w @ np.abs(z)))


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("up", [10, 18, 21, 22, 23, 24, 25, 26, 27, 28, 30, 34, 40, 60, 90])
@pytest.mark.parametrize("kind", ["ties", "two levels", "rising", "falling below"])
def test_scores_of_any_size(kind, up, name):
    # scores of 2^up and more that are whole in binary32, ties among them; in other rows of the same warps minus that, zero and small ones
    dtype = TYPES[name][0]
    n = 700
    q, cache, table, lengths, _ = winner_of(n, 0, 0, q_heads=5, dtype=dtype)
    code = np.full(n, 7)
    if kind == "two levels":
        code[np.random.default_rng(up).random(n) < 0.5] = 6
    elif kind == "rising":
        code = np.arange(n) * 8 // n  # 0 to 7
    elif kind == "falling below":
        code = np.where(np.arange(n) < 40, 7, -np.arange(n) % 8)
    at = torch.arange(n, device="cuda")
    cache.k[at // 32, 0, at % 32, 0] = torch.from_numpy(code & 15).to(torch.uint8).cuda()
    q[0, 0, :, 0] = torch.tensor([1.0, -1.0, 0.0, 2.0 ** -8, 1.5])
    rows = list(rows_of(q, cache, table, lengths, 2.0 ** up))
    check_rows(*run(q, cache, table, lengths, scale=2.0 ** up), rows, BITS[name])
    # the same scores from large queries and keys, where the type holds them
    half = min(up // 2, 12 if name == "f16" else 60)
    q *= 2.0 ** half
    cache.k_scales[..., 0] *= 2.0 ** half
    check_rows(*run(q, cache, table, lengths, scale=2.0 ** (up - 2 * half)), rows, BITS[name])


@pytest.mark.parametrize("scales", [[0.0, 2.0 ** 120], [2.0 ** 120, 0.0], [0.0, 2.0 ** 60, 1.0], [2.0 ** -70, 2.0 ** 60], [2.0 ** 60, 2.0 ** -70],
                                    [0.0, 2.0 ** 96, 0.0, 2.0 ** 124], [2.0 ** -75, 1.0, 2.0 ** 90]])
@pytest.mark.parametrize("n", [70, 700, 20000])
@pytest.mark.parametrize("offsets", [False, True])
def test_values_that_change_their_size_along_a_sequence(n, scales, offsets):
    # the weights of all positions count, whatever was met first and by whom
    q, cache, table, lengths, _ = winner_of(n, 0, 0, q_heads=3)
    cache.k[..., 0] = torch.from_numpy(np.random.default_rng(n).integers(0, 16, cache.k.shape[:-1]).astype(np.uint8)).cuda()
    at = torch.arange(n, device="cuda")
    size = torch.tensor(scales, device="cuda")[at * len(scales) // n].to(torch.bfloat16)
    cache.v_scales[at // 32, 0, at % 32, :, 0] = size[:, None]
    cache.v_scales[at // 32, 0, at % 32, :, 1] = (size[:, None] if offsets else 0 * size[:, None])
    q[0, 0, :, 0] = torch.tensor([0.0, 0.25, -1.0])
    check_rows(*run(q, cache, table, lengths, scale=1.0), rows_of(q, cache, table, lengths, 1.0), 8)


def test_the_largest_values_average_to_themselves():
    q, cache, table, lengths = problem(4, [30000, 64], 1, 2, 1, 64, 64, 64)
    cache.v_scales[..., 0], cache.v_scales[..., 1] = 0, torch.finfo(torch.bfloat16).max
    out = run(q, cache, table, lengths)[0]
    assert bool((out.double() >= torch.finfo(torch.bfloat16).max * (1 - 2.0 ** -7)).all()) and bool(torch.isfinite(out.float()).all())


@pytest.mark.parametrize("name,scales", [("bf16", [0.0, 2.0 ** 90]), ("bf16", [2.0 ** 90, 0.0]), ("bf16", [2.0 ** -70, 2.0 ** 20]),
                                         ("bf16", [1.0, 2.0 ** -60]), ("f16", [0.0, 64.0]), ("f16", [64.0, 2.0 ** -14])])
@pytest.mark.parametrize("far", [0, 300, 699])
def test_large_scores_beside_scales_of_any_size(name, scales, far):
    # scores of 0, then of 2^30 and more from position `far` on; values of one size and then of another
    dtype = TYPES[name][0]
    q, cache, table, lengths, _ = winner_of(700, 0, 0, q_heads=5, dtype=dtype)
    at = torch.arange(700, device="cuda")
    cache.k[at // 32, 0, at % 32, 0] = torch.where(at >= far, 7, 0).to(torch.uint8)
    cache.v_scales[..., 1] = 0
    for part, scale in zip((at < 350, at >= 350), scales):
        cache.v_scales[at[part] // 32, 0, at[part] % 32, :, 0] = scale
    q[0, 0, :, 0] = torch.tensor([1.0, -1.0, 0.0, 2.0 ** -28, 1.5])
    rows = [r for r in rows_of(q, cache, table, lengths, 2.0 ** 30) if np.any(r[1])]
    assert rows
    check_rows(*run(q, cache, table, lengths, scale=2.0 ** 30), rows, BITS[name])


@pytest.mark.parametrize("key,query", [(2.0 ** 123, 2.0 ** -123), (2.0 ** 100, 2.0 ** -99), (2.0 ** -110, 2.0 ** 112), (2.0 ** -20, 2.0 ** 21)])
@pytest.mark.parametrize("dim", [64, 256])
def test_queries_and_keys_of_any_size(key, query, dim):
    # powers of two that cancel, or nearly so, in the scores
    q, cache, table, lengths = problem(dim, [300, 31], 2, 6, 2, dim, 32, 32)
    cache.k_scales[..., 0], cache.k_scales[..., 1] = 2.0 ** -4, cache.k_scales[..., 1].clamp(-1, 1) * 0.25  # keys up to 3 / 4
    cache.k_scales *= key
    q = (q.float() * query).to(q.dtype)
    out, lse = run(q, cache, table, lengths)
    check_rows(out, lse, rows_of(q, cache, table, lengths, dim ** -0.5), 8)


def test_the_debug_build_declines_no_access_over_values_of_every_size(bq_lib):
    with _lib.use_library(build.build_debug_library()):
        codec.take_index_errors()
        test_rows_of_scales_of_any_size(120)
        test_large_values_of_no_weight("bf16", 90, 500)
        test_every_position_counts_once(SHARES[5])
        test_every_position_counts_once(SHARES[7])
        torch.cuda.synchronize()
        assert codec.take_index_errors() == 0
