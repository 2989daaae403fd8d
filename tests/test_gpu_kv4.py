"""The 4-bit cache against its definition: rows written and read bit for bit (numpy's binary32
arithmetic), attention in 64 bits on the values that the codes stand for.

Tolerance of attention. x_j = scale * <q, k_j> comes from sums of a group's q * (code + b), b an exact
offset of at most 144 that is taken off again: at most group + 2 terms of at most 160 max|q| in
16-column steps, each truncated once at 2^-23 of the largest of sum and terms. That is at most
E = scale * sum over groups of s * (group / 16 + 2) * 17 * 2^-23 * 160 * (max|q| + |sum q| so far), plus
(head_dim + 8) * 2^-23 * scale * sum |q| (|s code| + |offset|) for the rest. A change of every x_j by
at most E changes a softmax weight by a factor within exp(2 E) and lse by E. Weights times a scale are
rounded to FP16 (2^-11 relative, at least 2^-24 of the largest): 2^-11 max|v - offset|; exp, the sums over n positions
and the joins add at most (n / 16 + 64) * 2^-23 of sum |w v|. The output is rounded once.
"""
import math

import numpy as np
import pytest
import torch

from block_quantized_wire_gb300 import _lib, attention, build, codec, kv4
from tests.helpers import Guarded

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (torch.bfloat16, 8), "f16": (torch.float16, 11)}


# ---------------------------------------------------------------- write and read
def quantized(x, group):
    """Rows [..., dim] -> packed codes, pairs [..., groups, 2], and values, with numpy's binary32."""
    v = x.float().cpu().numpy().reshape(*x.shape[:-1], -1, group)

    def rounded(a):
        return torch.from_numpy(np.asarray(a, np.float32)).to(x.dtype)
    with np.errstate(all="ignore"):
        lo, hi = v.min(-1), v.max(-1)
        s = rounded((hi - lo) / np.float32(15))
        bad = ~np.isfinite(s.float().numpy())
        s32 = np.where(bad, np.float32("nan"), s.float().numpy())
        z = rounded((lo + np.float32(4) * s32) + np.float32(4) * s32)
        z32 = np.where(bad, np.float32("nan"), z.float().numpy())
        code = np.clip(np.rint((v - z32[..., None]) / s32[..., None]), -8, 7)
        code = np.where(s32[..., None] > 0, code, 0).astype(np.int64)
        value = rounded(code.astype(np.float32) * s32[..., None] + z32[..., None]).reshape(x.shape)
    code = code.reshape(x.shape)
    packed = ((code[..., 0::2] & 15) | ((code[..., 1::2] & 15) << 4)).astype(np.uint8)
    pairs = torch.stack([torch.from_numpy(s32), torch.from_numpy(z32)], dim=-1).to(x.dtype)
    return packed, pairs, value


def hard_rows(rng, tokens, heads, dim, group, dtype):
    """Rows of every scale; groups of zeros, constants, ties, one outlier, the smallest and the largest values, infinities and
    NaN."""
    x = rng.standard_normal((tokens, heads, dim)) * 10.0 ** rng.uniform(-4, 3, (tokens, heads, 1))
    x += rng.standard_normal((tokens, heads, 1)) * (rng.random((tokens, heads, 1)) < 0.3) * 50
    big = 3.38e38 if dtype is torch.bfloat16 else 65504.0
    tiny = 2.0 ** -133 if dtype is torch.bfloat16 else 2.0 ** -24
    g = x.reshape(-1, group)
    kinds = [lambda: np.zeros(group), lambda: np.full(group, 3.5), lambda: -np.zeros(group),
             lambda: rng.integers(-30, 31, group) * 0.25, lambda: np.r_[rng.integers(0, 31, group - 2) * 0.5, 0.0, 15.0],
             lambda: np.r_[rng.standard_normal(group - 1), 1e4], lambda: rng.integers(0, 40, group) * tiny,
             lambda: rng.choice([big, -big, 0.0], group), lambda: rng.choice([big / 4, -big / 4, 1.0], group),
             lambda: np.r_[np.inf, rng.standard_normal(group - 1)], lambda: np.r_[rng.standard_normal(group - 1), -np.inf],
             lambda: np.r_[np.nan, rng.standard_normal(group - 1)], lambda: rng.standard_normal(group) * 1e-36,
             lambda: np.r_[rng.standard_normal(group // 2), np.full(group - group // 2, np.nan)]]
    for i in range(0, len(g), 5):
        g[i] = kinds[i // 5 % len(kinds)]()
    return torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()


def guarded_cache(pages, heads, page, dim, group, dtype, token_first=False):
    """A cache in guarded buffers; token_first: tokens before heads in memory."""
    guards, parts = [], []
    order = (pages, page, heads) if token_first else (pages, heads, page)
    for _ in range(2):
        for last, t, size in (((dim // 2,), torch.uint8, 1), ((dim // group, 2), dtype, 2)):
            g = Guarded(math.prod(order) * math.prod(last) * size)
            g.raw[:] = Guarded.SENTINEL
            view = g.view(t, (*order, *last))
            parts.append(view.transpose(1, 2) if token_first else view)
            guards.append(g)
    return kv4.Cache(*parts), guards


def same_bits(a, b):
    return torch.equal(a.contiguous().cpu().view(torch.int16), b.contiguous().cpu().view(torch.int16))


# tokens, heads, dim, group, page, token first, columns between rows
ROWS = [(1, 1, 64, 32, 16, False, 0), (1, 8, 128, 64, 64, False, 0), (37, 3, 192, 64, 10, True, 8),
        (500, 8, 128, 32, 64, False, 0), (130, 2, 256, 128, 1, False, 16), (65, 5, 64, 64, 100, True, 0),
        (333, 1, 256, 32, 24, False, 0), (200, 7, 128, 128, 32, True, 64), (2000, 4, 192, 32, 7, False, 0),
        (90, 2, 256, 64, 48, True, 8)]


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("shape", ROWS)
def test_write_and_read_are_bit_exact(shape, name, wide):
    tokens, heads, dim, group, page, token_first, pad = shape
    dtype = TYPES[name][0]
    rng = np.random.default_rng(tokens + dim + group)
    pages = -(-tokens // page) + 3
    cache, guards = guarded_cache(pages, heads, page, dim, group, dtype, token_first)
    at = torch.from_numpy(rng.permutation(pages * page)[:tokens])
    if tokens > 3:
        at[1], at[2], at[-1] = -1, pages * page, -2 ** 31  # no slots of this cache
    held = (at >= 0) & (at < pages * page)
    slots = (at if wide else at.int()).cuda()
    both = torch.full((tokens, 2 * heads, dim + pad), float("nan"), dtype=dtype, device="cuda")
    both[..., :dim] = hard_rows(rng, tokens, 2 * heads, dim, group, dtype)
    k, v = both[:, :heads, :dim], both[:, heads:, :dim]  # as one projection gives them
    kv4.write(k, v, slots, cache)
    page_of, place = at[held] // page, at[held] % page
    untouched = torch.ones(pages, page, dtype=torch.bool)
    untouched[page_of, place] = False
    for rows, codes, pairs in ((k, cache.k, cache.k_scales), (v, cache.v, cache.v_scales)):
        want, want_pairs, value = quantized(rows[held.cuda()], group)
        got, got_pairs = codes.cpu()[page_of, :, place], pairs.cpu()[page_of, :, place]
        assert np.array_equal(got.numpy(), want)
        fine = ~torch.isnan(want_pairs.float())
        assert torch.equal(torch.isnan(got_pairs.float()), ~fine) and torch.equal(got_pairs[fine], want_pairs[fine])
        assert bool((codes.cpu().transpose(1, 2)[untouched] == Guarded.SENTINEL).all())
        assert bool((pairs.cpu().view(torch.int16).transpose(1, 2)[untouched] == -23131).all())  # 0xa5a5
    gk, gv = (Guarded(2 * tokens * heads * (dim + pad)) for _ in range(2))
    out = [g.view(dtype, (tokens, heads, dim + pad))[..., :dim] for g in (gk, gv)]
    kv4.read(cache, slots, *out)
    for rows, got in zip((k, v), out):
        value = quantized(rows, group)[2]
        value[~held] = 0
        fine = ~torch.isnan(value.float())
        got = got.cpu()
        assert torch.equal(torch.isnan(got.float()), ~fine) and torch.equal(got[fine], value[fine])
    assert all(g.bands_intact() for g in (*guards, gk, gv))
    if pad:
        assert bool((gk.view(torch.uint8).view(tokens, heads, -1)[..., 2 * dim:] == Guarded.SENTINEL).all())


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("group", [32, 64, 128])
def test_a_value_is_off_by_half_a_step(name, group):
    # x - (s c + z) is at most half a step and what the rounding of s and z to 16 bits costs at the ends of
    # the range: 15 steps times 2^-p of s, and 2^-p of the offset; and one rounding of the value
    dtype, p = TYPES[name]
    rng = np.random.default_rng(group)
    x = torch.from_numpy(rng.standard_normal((50, 2, 256)).astype(np.float32) + 3).to(dtype).cuda()
    cache = kv4.empty_cache(50, 2, 1, 256, group, dtype)
    slots, out = torch.arange(50, device="cuda"), torch.empty_like(x)
    kv4.write(x, x, slots, cache)
    kv4.read(cache, slots, out, torch.empty_like(x))
    v = x.double().view(50, 2, -1, group)
    step = (v.amax(-1, keepdim=True) - v.amin(-1, keepdim=True)) / 15
    bound = step * (0.5 + 16 * 2.0 ** -p) * (1 + 2.0 ** -p) + 2.0 ** -p * v.abs().amax(-1, keepdim=True) * 2
    assert bool(((out.double().view_as(v) - v).abs() <= bound).all())


def test_write_rows_aligned_to_16_but_not_32_bytes():
    rng = np.random.default_rng(3)
    base = torch.from_numpy(rng.standard_normal(40 * 2 * 128 + 8).astype(np.float32)).to(torch.bfloat16).cuda()
    x = base[8:].view(40, 2, 128)
    cache = kv4.empty_cache(3, 2, 16, 128)
    slots = torch.arange(40, device="cuda", dtype=torch.int32)
    kv4.write(x, base[:-8].view(40, 2, 128), slots, cache)
    out = torch.empty(2, 40 * 2 * 128 + 8, dtype=torch.bfloat16, device="cuda")
    k, v = out[0, 8:].view(40, 2, 128), out[1, 8:].view(40, 2, 128)
    kv4.read(cache, slots, k, v)
    assert same_bits(k, quantized(x, 64)[2]) and same_bits(v, quantized(base[:-8].view(40, 2, 128), 64)[2])


def test_a_row_given_to_every_head_and_token():
    x = torch.randn(1, 1, 128, device="cuda").to(torch.float16)
    cache = kv4.empty_cache(2, 4, 8, 128, 32, torch.float16)
    slots = torch.arange(16, device="cuda")
    kv4.write(x.expand(16, 4, 128), x.expand(16, 4, 128), slots, cache)
    k, v = (torch.empty(16, 4, 128, dtype=torch.float16, device="cuda") for _ in range(2))
    kv4.read(cache, torch.zeros_like(slots), k, v)  # one slot read by all
    want = quantized(x, 32)[2].expand(16, 4, 128)
    assert same_bits(k, want) and same_bits(v, want)


# ---------------------------------------------------------------- attention
def block_cache(pages, heads, page, dim, group, dtype):
    """All four arrays of a page in one block of memory."""
    row, row_s = dim // 2, 4 * (dim // group)
    sizes = [heads * page * n for n in (row, row, row_s, row_s)]
    starts = [sum((s + 15) // 16 * 16 for s in sizes[:i]) for i in range(5)]
    block = torch.zeros((pages, starts[4]), dtype=torch.uint8, device="cuda")

    def part(i, last, t):
        flat = block[:, starts[i]:starts[i] + sizes[i]]
        flat = flat if t is torch.uint8 else block.view(t)[:, starts[i] // 2:(starts[i] + sizes[i]) // 2]
        inner = math.prod(last)
        return flat.as_strided((pages, heads, page, *last), (flat.stride(0), page * inner, inner, *((last[1], 1) if len(last) > 1
                                                                                                      else (1,))),
                               flat.storage_offset())
    return kv4.Cache(part(0, (row,), torch.uint8), part(2, (dim // group, 2), dtype), part(1, (row,), torch.uint8),
                     part(3, (dim // group, 2), dtype))


def fill(rng, cache, spread=0.2):
    """All sixteen codes, scales around 0.4, offsets around 1."""
    for codes, pairs in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
        codes.copy_(torch.from_numpy(rng.integers(0, 256, codes.shape, dtype=np.uint8)))
        s = np.exp(rng.standard_normal(pairs.shape[:-1]) * spread) * 0.2
        z = rng.standard_normal(pairs.shape[:-1])
        pairs.copy_(torch.from_numpy(np.stack([s, z], -1).astype(np.float32)))


def values64(codes, pairs, table, lengths, page):
    """[positions, heads, dim] in 64 bits for each sequence, and which positions have a page."""
    codes, pairs, table = codes.cpu().numpy(), pairs.double().cpu().numpy(), table.cpu().numpy()
    out = []
    for b, length in enumerate(lengths):
        j = np.arange(length)
        at = table[b, j // page] if length else np.zeros(0, np.int64)
        there = (at >= 0) & (at < codes.shape[0])
        at = np.where(there, at, 0)
        c, p = codes[at, :, j % page].astype(np.int64), pairs[at, :, j % page]
        c = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], 2 * c.shape[-1])
        c = np.where(c > 7, c - 16, c)
        group = c.shape[-1] // p.shape[-2]
        p = np.repeat(p, group, axis=-2)
        out.append((c * p[..., 0] + p[..., 1], p[..., 0], np.abs(p[..., 1]), there))
    return out


def reference(q, cache, table, lengths, scale, window, p):
    """out, lse and their bounds."""
    batch, n_q, q_heads, dim = q.shape
    lens = [max(0, min(int(n), table.shape[1] * cache.page)) for n in lengths.cpu()]
    ks, vs = (values64(c, s, table, lens, cache.page) for c, s in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)))
    out, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    bound, bound_lse = np.zeros(q.shape), np.zeros(q.shape[:3])
    q64 = q.double().cpu().numpy()
    share = q_heads // cache.heads
    for b, length in enumerate(lens):
        (k, ksc, kz, there), (v, vsc, vz, _) = ks[b], vs[b]
        for i in range(n_q):
            hi = length - n_q + i + 1
            lo = max(0, hi - window) if window else 0
            at = np.arange(lo, max(lo, hi))
            at = at[there[at]]
            if not len(at):
                continue
            for h in range(q_heads):
                g = h // share
                row = q64[b, i, h]
                x = scale * (k[at, g] @ row)
                part = np.abs(np.cumsum(row.reshape(-1, cache.group), -1)).max(-1) + np.abs(row).max()
                e = abs(scale) * ((ksc[at, g].reshape(len(at), -1, cache.group)[..., 0] * part).sum(-1).max()
                                  * (cache.group / 16 + 2) * 17 * 160
                                  + (dim + 8) * (np.abs(row) * (np.abs(k[at, g]) + 2 * kz[at, g])).sum(-1).max()) * 2.0 ** -23
                e += 4 * 2.0 ** -23 * np.abs(x).max()
                top = x.max()
                w = np.exp(x - top)
                total = w.sum()
                lse[b, i, h] = top + np.log(total)
                w /= total
                out[b, i, h] = w @ v[at, g]
                steps = (len(at) / 16 + 64) * 2.0 ** -23
                bound_lse[b, i, h] = e + steps + 4 * 2.0 ** -23 * abs(lse[b, i, h])
                mag = w @ (np.abs(v[at, g]) + vz[at, g])
                away = np.abs(v[at, g] - out[b, i, h]).max(0)
                bound[b, i, h] = ((math.exp(2 * e) - 1) * away + 2.0 ** -11 * (w @ (8 * vsc[at, g])) + steps * mag
                                  + 2.0 ** -24 * 8 * vsc[at, g].max(0)
                                  + 2.0 ** -p * np.abs(out[b, i, h])) * 1.01 + 2.0 ** -25
    return out, lse, bound, bound_lse


def table_of(rng, lengths, page, width, pages):
    """Pages anywhere, -1 past a sequence's own."""
    need = [-(-max(0, min(int(n), width * page)) // page) for n in lengths]
    assert sum(need) <= pages
    order = rng.permutation(pages)
    table = np.full((len(lengths), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table).cuda()


def check(out, lse, want, cache=None):
    o, l, bound, bound_lse = want
    got = out.double().cpu().numpy()
    err = np.abs(got - o) - bound
    assert np.all(np.isfinite(got)) and np.all(err <= 0), (float(err.max()), np.argwhere(err > 0)[:4])
    if lse is not None:
        got = lse.double().cpu().numpy()
        assert np.array_equal(np.isneginf(got), np.isneginf(l))
        fine = np.isfinite(l)
        err = np.abs(got[fine] - l[fine]) - bound_lse[fine]
        assert np.all(err <= 0), float(err.max())


def run(q, cache, table, lengths, with_lse=True, pad=0, workspace=None, **more):
    """attend into guarded outputs with garbage in the workspace."""
    g = Guarded(2 * q.numel() // q.shape[-1] * (q.shape[-1] + pad))
    out = g.view(q.dtype, (*q.shape[:3], q.shape[-1] + pad))[..., :q.shape[-1]]
    gl = Guarded(4 * q.numel() // q.shape[-1])
    lse = gl.view(torch.float32, q.shape[:3]) if with_lse else None
    if workspace is None:
        workspace = kv4.empty_workspace(q, cache)
        workspace.fill_(255)  # NaN
    kv4.attend(q, cache, table, lengths, out, workspace, lse=lse, **more)
    assert g.bands_intact() and gl.bands_intact()
    if pad:
        assert bool((g.view(torch.uint8).view(-1, 2 * (q.shape[-1] + pad))[:, 2 * q.shape[-1]:] == Guarded.SENTINEL).all())
    return out, lse


# lengths, queries, q heads, heads, dim, group, page, window
ATTEND = [([1], 1, 1, 1, 64, 32, 16, 0), ([2], 1, 8, 1, 128, 64, 64, 0), ([15, 16, 17], 1, 8, 2, 128, 128, 16, 0),
          ([0, 1, 40, 0], 1, 4, 4, 128, 32, 64, 0), ([500], 1, 64, 8, 128, 64, 64, 0), ([33, 700, 5], 1, 15, 3, 192, 64, 10, 0),
          ([200, 31], 1, 12, 1, 256, 128, 1, 0), ([3000], 1, 8, 1, 128, 64, 64, 0), ([3000, 10], 1, 16, 1, 64, 64, 100, 0),
          ([129, 64], 4, 16, 2, 128, 128, 32, 0), ([3, 1, 0, 70], 5, 6, 2, 64, 32, 7, 0), ([260], 8, 12, 1, 256, 32, 48, 0),
          ([90, 17], 3, 32, 2, 128, 32, 16, 0), ([400, 30], 1, 8, 2, 128, 64, 32, 16), ([400, 3, 77], 2, 10, 2, 192, 32, 24, 1),
          ([1000, 250], 6, 4, 1, 256, 64, 16, 100), ([513] * 40, 1, 8, 4, 64, 32, 16, 0), ([5000], 1, 5, 1, 64, 64, 8, 0),
          ([2049, 1], 1, 7, 1, 256, 128, 64, 0), ([300, 290], 40, 4, 1, 64, 64, 64, 0)]


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("shape", ATTEND)
def test_attend(shape, name):
    lens, n_q, q_heads, heads, dim, group, page, window = shape
    dtype, p = TYPES[name]
    rng = np.random.default_rng(sum(lens) + dim + q_heads)
    width = -(-max(lens) // page) + 2
    pages = sum(-(-n // page) for n in lens) + 2
    cache = (block_cache if name == "f16" else kv4.empty_cache)(pages, heads, page, dim, group, dtype)
    fill(rng, cache)
    table = table_of(rng, lens, page, width, pages)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.from_numpy(rng.standard_normal((len(lens), n_q, q_heads, dim)).astype(np.float32)).to(dtype).cuda()
    out, lse = run(q, cache, table, lengths, pad=8 if q_heads % 2 else 0, window=window)
    check(out, lse, reference(q, cache, table, lengths, dim ** -0.5, window, p))
    again, lse_again = run(q, cache, table, lengths, window=window)
    assert same_bits(out, again) and torch.equal(lse, lse_again)  # a call repeated gives the same bits
    plain, _ = run(q, cache, table, lengths, with_lse=False, window=window)
    assert same_bits(out, plain)


@pytest.mark.parametrize("name", list(TYPES))
def test_what_a_query_does_not_see_is_not_looked_at(name):
    # rows behind a sequence's end, before its window, and in pages that the table does not name hold NaN
    dtype, p = TYPES[name]
    rng = np.random.default_rng(5)
    lens, page, window, n_q = [77, 200, 9], 16, 50, 2
    cache = kv4.empty_cache(40, 2, page, 128, 32, dtype)
    fill(rng, cache)
    table = table_of(rng, lens, page, 20, 40)
    named = torch.zeros(40, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(max(0, n - n_q + 1 - window), n):
            named[table[b, j // page].item(), j % page] = True
    for t in (cache.k_scales, cache.v_scales):
        t.transpose(1, 2)[~named.cuda()] = float("nan")
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.from_numpy(rng.standard_normal((3, n_q, 4, 128)).astype(np.float32)).to(dtype).cuda()
    want = reference(q, cache, table, lengths, 128 ** -0.5, window, p)
    check(*run(q, cache, table, lengths, window=window), want)
    # columns before the window and past the end may name anything
    wild = table.clone()
    for b, n in enumerate(lens):
        wild[b, -(-n // page):] = 2 ** 31 - 1
        wild[b, :max(0, n - n_q + 1 - window) // page] = -2 ** 31
    check(*run(q, cache, wild, lengths, window=window), want)


def test_the_first_queries_see_less():
    # a NaN in the last position reaches the last query only
    rng = np.random.default_rng(6)
    cache = kv4.empty_cache(4, 1, 16, 64, 32)
    fill(rng, cache)
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([37], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 3, 2, 64, device="cuda").to(torch.bfloat16)
    clean, _ = run(q, cache, table, lengths)
    for t in (cache.k_scales, cache.v_scales):
        saved = t[3, 0, 4].clone()
        t[3, 0, 4] = float("nan")
        out, _ = run(q, cache, table, lengths)
        t[3, 0, 4] = saved
        assert same_bits(out[:, :2], clean[:, :2]) and bool(torch.isnan(out[:, 2]).any())


@pytest.mark.parametrize("page", [16, 10])
def test_pages_outside_the_cache_take_part_in_nothing(page):
    rng = np.random.default_rng(7)
    cache = kv4.empty_cache(12, 2, page, 128, 64)
    fill(rng, cache)
    lengths = torch.tensor([100, 64, 30], dtype=torch.int32, device="cuda")
    table = table_of(rng, [40, 30, 20], page, 11, 12)
    table[0, 3:7] = torch.tensor([-1, 12, 2 ** 31 - 1, -2 ** 31])
    table[0, 7:10] = table[0, :3]  # a page named twice
    table[1, 1] = -5
    table[2] = -1
    q = torch.randn(3, 1, 8, 128, device="cuda").to(torch.bfloat16)
    out, lse = run(q, cache, table, lengths)
    check(out, lse, reference(q, cache, table, lengths, 128 ** -0.5, 0, 8))
    assert not out[2].any() and bool(torch.isneginf(lse[2]).all())


def test_lengths_outside_the_table():
    rng = np.random.default_rng(8)
    cache = kv4.empty_cache(6, 1, 16, 64, 64)
    fill(rng, cache)
    table = table_of(rng, [48, 48], 16, 3, 6)
    q = torch.randn(2, 1, 4, 64, device="cuda").to(torch.bfloat16)
    for a, b in ((-1, 1000), (-2 ** 31, 2 ** 31 - 1)):
        lengths = torch.tensor([a, b], dtype=torch.int32, device="cuda")
        out, lse = run(q, cache, table, lengths)
        check(out, lse, reference(q, cache, table, lengths, 0.125, 0, 8))
        assert not out[0].any()
    none = table[:, :0]
    out, lse = run(q, cache, none, lengths)
    assert not out.any() and bool(torch.isneginf(lse).all())
    empty = kv4.empty_cache(0, 1, 16, 64, 64)
    out, lse = run(q, empty, table, lengths)
    assert not out.any()


@pytest.mark.parametrize("name", list(TYPES))
def test_values_of_very_different_sizes(name):
    # a group a million times larger than its neighbour, values from token to token too; sharp and flat softmaxes
    dtype, p = TYPES[name]
    rng = np.random.default_rng(9)
    cache = kv4.empty_cache(30, 1, 32, 128, 32, dtype)
    fill(rng, cache)
    cache.v_scales[:, :, :, 1] *= 2.0 ** -12
    cache.v_scales[:, :, :, 2] *= 2.0 ** 8
    cache.v_scales *= torch.from_numpy(2.0 ** rng.integers(-2, 3, (30, 1, 32, 1, 1))).to(dtype).cuda()
    lens = [900, 20]
    table = table_of(rng, lens, 32, 29, 30)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.from_numpy(rng.standard_normal((2, 1, 8, 128)).astype(np.float32)).to(dtype).cuda()
    for scale in (1.0, 0.01, 0.0, -0.2):
        check(*run(q, cache, table, lengths, scale=scale), reference(q, cache, table, lengths, scale, 0, p))


def test_a_tie_of_large_scores_and_a_single_winner():
    cache = kv4.empty_cache(64, 1, 16, 64, 64)
    k = torch.zeros(1024, 1, 64, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(1024, 1, 64, device="cuda").to(torch.bfloat16)
    k[:, 0, 0] = 100.0
    slots = torch.arange(1024, device="cuda")
    kv4.write(k, v, slots, cache)
    table = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    lengths = torch.tensor([1024], dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 1, 2, 64, device="cuda", dtype=torch.bfloat16)
    q[0, 0, 0, 0], q[0, 0, 1, 0] = 50.0, -50.0
    check(*run(q, cache, table, lengths), reference(q, cache, table, lengths, 0.125, 0, 8))
    k[700, 0, 0] = 120.0
    kv4.write(k, v, slots, cache)
    out, lse = run(q, cache, table, lengths)
    check(out, lse, reference(q, cache, table, lengths, 0.125, 0, 8))


def test_a_long_cache_past_31_bits_of_bytes():
    # page strides that pass 2^31 within a few pages, and slots past 2^31 in another cache
    pages, heads, page = 70000, 8, 64
    cache = kv4.empty_cache(pages, heads, page, 128, 128)
    assert cache.k.numel() > 2 ** 31
    rng = np.random.default_rng(10)
    table = torch.tensor([[69999, 5, 66000, 40000]], dtype=torch.int32, device="cuda")
    pos = torch.arange(250, device="cuda")[None]
    k, v = (torch.from_numpy(rng.standard_normal((250, heads, 128)).astype(np.float32)).to(torch.bfloat16).cuda()
            for _ in range(2))
    slots = kv4.slots(table, pos, page)[0]
    kv4.write(k, v, slots, cache)
    back = [torch.empty_like(k) for _ in range(2)]
    kv4.read(cache, slots, *back)
    assert same_bits(back[0], quantized(k, 128)[2]) and same_bits(back[1], quantized(v, 128)[2])
    small = kv4.empty_cache(4, heads, page, 128, 128)
    kv4.write(k, v, torch.arange(250, device="cuda"), small)
    q = torch.randn(1, 1, 16, 128, device="cuda").to(torch.bfloat16)
    lengths = torch.tensor([250], dtype=torch.int32, device="cuda")
    far, _ = run(q, cache, table, lengths)
    near, _ = run(q, small, torch.arange(4, dtype=torch.int32, device="cuda")[None], lengths)
    assert same_bits(far, near)


def test_slots_past_31_bits():
    cache = kv4.empty_cache(40000, 1, 65536, 64, 64)  # 2.6e9 slots
    x = torch.randn(4, 1, 64, device="cuda").to(torch.bfloat16)
    slots = torch.tensor([2 ** 31 + 5, 40000 * 65536 - 1, 3, 40000 * 65536], device="cuda")
    out = [torch.empty_like(x) for _ in range(2)]
    kv4.write(x, x, slots, cache)
    kv4.read(cache, slots, *out)
    want = quantized(x, 64)[2]
    want[3] = 0
    assert same_bits(out[0], want) and same_bits(out[1], want)


# ---------------------------------------------------------------- together, and beside other work
def test_a_captured_step_follows_its_inputs():
    # write and attend captured once; replayed with other rows, tables and lengths
    rng = np.random.default_rng(11)
    cache, table = kv4.empty_cache(20, 2, 16, 128, 64), torch.zeros((2, 9), dtype=torch.int32, device="cuda")
    lengths = torch.zeros(2, dtype=torch.int32, device="cuda")
    fill(rng, cache)
    q, k, v = (torch.zeros(2, 1, h, 128, device="cuda", dtype=torch.bfloat16) for h in (8, 2, 2))
    out, ws = torch.zeros_like(q), kv4.empty_workspace(q, cache)

    def step():
        kv4.write(k[:, 0], v[:, 0], kv4.slots(table, lengths[:, None] - 1, 16)[:, 0], cache)
        kv4.attend(q, cache, table, lengths, out, ws)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([30, 128], [31, 1], [1, 140], [0, 7]):
        table.copy_(table_of(rng, lens, 16, 9, 20))
        lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        for t in (q, k, v):
            t.copy_(torch.randn_like(t, dtype=torch.float32))
        graph.replay()
        torch.cuda.synchronize()
        check(out, None, reference(q, cache, table, lengths, 128 ** -0.5, 0, 8))


def test_calls_on_several_streams_at_once():
    rng = np.random.default_rng(12)
    cache = kv4.empty_cache(200, 2, 32, 128, 32)
    fill(rng, cache)
    lens = [3000, 1500, 40]
    table = table_of(rng, lens, 32, 95, 200)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qs = [torch.randn(3, 1, 16, 128, device="cuda").to(torch.bfloat16) for _ in range(4)]
    want = [run(q, cache, table, lengths)[0] for q in qs]
    outs, wss = [torch.empty_like(q) for q in qs], [kv4.empty_workspace(q, cache) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        for q, out, ws, s in zip(qs, outs, wss, streams):
            kv4.attend(q, cache, table, lengths, out, ws, stream=s)
    torch.cuda.synchronize()
    assert all(same_bits(a, b) for a, b in zip(outs, want))


def test_the_debug_build_declines_no_access(bq_lib):
    with _lib.use_library(build.build_debug_library()):
        codec.take_index_errors()
        for i in (0, 2, 4, 6):
            test_write_and_read_are_bit_exact(ROWS[i], "bf16", bool(i & 2))
        for i in (0, 3, 5, 9, 11, 13, 15, 18):
            test_attend(ATTEND[i], "f16")
        test_what_a_query_does_not_see_is_not_looked_at("bf16")
        test_pages_outside_the_cache_take_part_in_nothing(16)
        test_pages_outside_the_cache_take_part_in_nothing(10)
        test_lengths_outside_the_table()
        torch.cuda.synchronize()
        assert codec.take_index_errors() == 0


# ---------------------------------------------------------------- a layer's attention
def dequantized(pair):
    q, s = (t.cpu() for t in pair)
    q = q.to(torch.int64)
    code = torch.stack([q & 15, q >> 4], dim=-1).flatten(-2)
    code = torch.where(code > 7, code - 16, code)
    return code.double() * s.double().repeat_interleave(code.shape[-1] // s.shape[-1], dim=-1)


def a_layer(mode, n_ranks=2, steps=3):
    torch.manual_seed(13)
    rng = np.random.default_rng(13)
    batch, hidden, q_heads, heads, dim, page = 4, 512, 4, 2, 64, 16
    ranks, caches, wss = [], [], []
    for _ in range(n_ranks):
        qkv = (torch.randn((q_heads + 2 * heads) * dim, hidden, device="cuda") * hidden ** -0.5).to(torch.bfloat16)
        o = (torch.randn(hidden, q_heads * dim, device="cuda") * (q_heads * dim) ** -0.5).to(torch.bfloat16)
        ranks.append(attention.quantize_heads(q_heads, heads, qkv, o))
        caches.append(kv4.empty_cache(30, heads, page, dim, 32))
    table = table_of(rng, [90] * batch, page, 6, 30)
    lengths = torch.tensor([5, 0, 33, 60], dtype=torch.int32, device="cuda")
    for c in caches:
        fill(rng, c)
    xs = [torch.randn(batch, hidden, device="cuda").to(torch.bfloat16) for _ in range(steps)]
    return ranks, caches, table, lengths, xs


@pytest.mark.parametrize("mode", ["", "i8_a2a", "mx_a2a", "i8_ring"])
def test_decode_steps_over_ranks(mode):
    ranks, caches, table, lengths, xs = a_layer(mode)
    w = [(dequantized(r.qkv), dequantized(r.out)) for r in ranks]
    for x in xs:
        lengths += 1
        out = torch.cat(attention.decode_layer(x, ranks, caches, table, lengths, mode)).double().cpu()
        want = torch.zeros_like(out)
        for (qkv, o), cache, rank in zip(w, caches, ranks):
            # keys and values as the cache now holds them; the queries rounded to BF16 as the products give them
            rows = (x.double().cpu() @ qkv[:rank.q_heads * 64].T).to(torch.bfloat16).view(4, 1, rank.q_heads, 64)
            want += torch.from_numpy(reference(rows, cache, table, lengths, 0.125, 0, 8)[0]).view(4, -1) @ o.T
        # BF16 roundings of queries, heads, parts and sum (2^-8 each, five deep), and, per wire hop, a payload step of
        # amax / 127 / 2 (INT8) or 2^-4 of the value (E4M3)
        amax = float(want.abs().max())
        wire = {"": 0.0, "i8_a2a": 3 / 254, "i8_ring": 2 / 254, "mx_a2a": 2 / 16}[mode]
        assert float((out - want).abs().max()) <= (5 * 2.0 ** -8 * 4 + wire * 2) * amax
        # the new row is in the cache: the last position's key is the product, to half a step of its codes
        slots = kv4.slots(table, lengths[:, None] - 1, 16)[:, 0]
        k, v = (torch.empty(4, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        kv4.read(caches[0], slots, k, v)
        fresh = (x.double().cpu() @ w[0][0][4 * 64:].T).view(4, 2, 2, 64)
        spread = fresh.amax(-1, keepdim=True) - fresh.amin(-1, keepdim=True)
        for got, new in ((k, fresh[:, 0]), (v, fresh[:, 1])):
            assert bool(((got.double().cpu() - new).abs() <= spread[:, 0].max() * (0.5 / 15 + 2.0 ** -6)).all())


def test_a_rotation_of_queries_and_keys_is_applied():
    ranks, caches, table, lengths, (x,) = a_layer("", n_ranks=1, steps=1)
    lengths += 1
    seen = []

    def negate(q, k, positions):
        seen.append(positions.clone())
        return -q, -k
    a = attention.decode_layer(x, ranks, caches, table, lengths, "", rotate=negate)[0]
    assert seen[0].tolist() == (lengths[:, None] - 1).tolist()
    slots = kv4.slots(table, lengths[:, None] - 1, 16)[:, 0]
    k, v = (torch.empty(4, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kv4.read(caches[0], slots, k, v)
    attention.decode_layer(x, ranks, caches, table, lengths, "")
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    kv4.read(caches[0], slots, k2, v2)
    assert same_bits(v, v2) and not same_bits(k, k2) and bool(torch.isfinite(a.float()).all())
