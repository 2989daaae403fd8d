"""Tight checks of attention over the 4-bit cache, beside the worst-case bounds of test_gpu_kv4: what an output may be off by
as a whole row, and values of which every position's share in the output is known exactly.

A row as a whole. The output is rounded once: at most 2^-p of each value, so at most 2^-p of the row's root mean square.
A weight times a scale is rounded to FP16, 2^-11, each token's by itself: these add up as independent errors do, to at most 2^-11 of
S = sqrt(sum_j (w_j |v_j|)^2), |v_j| the root mean square of (value - offset) and of the offset together. Scores: with q of about
N(0, 1) in head_dim <= 256 columns partial sums of q u (u <= 15) stay within 2^12, about 10 truncations a group of 2^-23 of
that, times a scale of at most 0.8 and head_dim ** -0.5: below 2^-11, again each token's by itself, so at most 2^-11 of S. Sums over positions
in binary32 add (n / 16 + 64) 2^-23 of sum_j w_j |v_j|."""
import numpy as np

BITS = {"bf16": 8, "f16": 11}


def decoded(codes, pairs):
    """Values and scales [..., head_dim] in 64 bits of codes [..., head_dim / 2] and pairs [..., groups, 2]."""
    c, p = codes.cpu().numpy().astype(np.int64), pairs.double().cpu().numpy()
    c = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], 2 * c.shape[-1])
    c = np.where(c > 7, c - 16, c)
    p = np.repeat(p, c.shape[-1] // p.shape[-2], axis=-2)
    return c * p[..., 0] + p[..., 1], p[..., 0], p[..., 1]


def seen(length, i, n_q, window):
    """The positions that query i of n_q sees in a sequence of `length` positions."""
    hi = length - n_q + i + 1
    return np.arange(max(0, hi - window) if window else 0, max(hi, 0))


def rows_of(q, cache, table, lengths, scale, window=0, drop=None):
    """For each query and head that sees something: its index, out and lse in 64 bits, what the checks need of its weights.
    drop(b, h, positions) gives positions whose values a planted mistake leaves out of the sum."""
    k, _, _ = decoded(cache.k, cache.k_scales)
    v, s, z = decoded(cache.v, cache.v_scales)
    q, table = q.double().cpu().numpy(), table.cpu().numpy()
    batch, n_q, q_heads, dim = q.shape
    for b, length in enumerate(int(n) for n in lengths.cpu()):
        for i in range(n_q):
            at = seen(length, i, n_q, window)
            if not len(at):
                continue
            page, place = table[b, at // cache.page], at % cache.page
            for h in range(q_heads):
                g = h * cache.heads // q_heads
                x = scale * (k[page, g, place] @ q[b, i, h])
                top = x.max()
                w = np.exp(x - top)
                total = w.sum()
                w /= total
                vs, ss, zs = v[page, g, place], s[page, g, place], z[page, g, place]
                kept = w.copy()
                if drop is not None:
                    kept[drop(b, h, at)] = 0
                yield (b, i, h), kept @ vs, top + np.log(total), w, vs, ss, zs


def rms(a):
    return np.sqrt(np.mean(np.square(a), axis=-1))


def row_error(out, row, p):
    """The error of one output row beside what the module's arithmetic allows it."""
    at, want, _, w, v, s, z = row
    size = rms(v - z) + rms(z)
    allowed = (2.0 ** -p * rms(want) + (2.0 ** -11 + 2.0 ** -11) * np.sqrt(np.sum(np.square(w * size)))
               + (len(w) / 16 + 64) * 2.0 ** -23 * (w @ size))
    return rms(out[at] - want) / allowed


def check_rows(out, lse, rows, p):
    """Every row within what is allowed; lse to 2^-11 and the roundings of a number of its size."""
    out = out.double().cpu().numpy() if hasattr(out, "cpu") else out
    for row in rows:
        error = row_error(out, row, p)
        assert error <= 1, (row[0], error)
        if lse is not None:
            assert abs(float(lse[row[0]]) - row[2]) <= 2.0 ** -11 + (len(row[3]) / 16 + 64) * 2.0 ** -23 + 2.0 ** -21 * abs(row[2])


# ---------------------------------------------------------------- every position's share known
def marked_codes(positions, dim):
    """Codes [positions, dim]: 7 in column j % dim of position j, 0 elsewhere."""
    code = np.zeros((positions, dim), np.int64)
    code[np.arange(positions), np.arange(positions) % dim] = 7
    return code


def shares(length, n_q, window, dim, drop=()):
    """[n_q, dim]: the mean of marked_codes over what each query sees; positions in `drop` are left out of the sum, not of
    the count: the mistake that a lost part of a value sum is."""
    out = np.zeros((n_q, dim))
    for i in range(n_q):
        at = seen(length, i, n_q, window)
        if len(at):
            out[i] = 7.0 * np.bincount(np.setdiff1d(at, drop) % dim, minlength=dim) / len(at)
    return out


def check_shares(out, want, p=11):
    """Sums of whole numbers, exact in binary32 below 2^24, times fl(1 / n): two roundings of 2^-24, one of 2^-p."""
    assert np.all(np.abs(out - want) <= want * (2.0 ** -p + 2.0 ** -22)), np.argwhere(np.abs(out - want) > want * 2.0 ** -p)[:4]
