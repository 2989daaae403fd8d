"""The operators of a key-value cache in 4 bits as measured: their cases, inputs, plain forms and exact values.

* ``write``    rows of keys and values quantized into the pages of a cache, and given back as the cache holds them
* ``read``     a cache's rows by slot, as 16-bit values
* ``attend``   attention of a few query tokens of each sequence over its pages

A row (one head of one token) is held as signed 4-bit codes with a scale and an offset for each group of columns:
value = code * scale + offset. ``run`` computes the operators with elementary torch operations in 32 bits (``own``
false) or with this repository's kernels (``own`` true). ``exact`` restates the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 64 requests: latency is what counts
        {"name": "write decode", "op": "write", "tokens": 64, "heads": 8, "dim": 128, "group": 64, "page": 64,
         "dtype": "bf16", "skip": False},
        # a prefill chunk, fine groups
        {"name": "write prefill", "op": "write", "tokens": 32768, "heads": 8, "dim": 128, "group": 32, "page": 64,
         "dtype": "bf16", "skip": False},
        # a padded batch (some tokens have no slot), pages of an odd size
        {"name": "write padded odd", "op": "write", "tokens": 1999, "heads": 5, "dim": 192, "group": 64, "page": 24,
         "dtype": "f16", "skip": True},
        # a shared prefix brought back for a prefill's attention
        {"name": "read prefix", "op": "read", "tokens": 65536, "heads": 8, "dim": 128, "group": 64, "page": 64,
         "dtype": "bf16", "skip": False},
        # a short prefix of narrow heads
        {"name": "read short odd", "op": "read", "tokens": 777, "heads": 3, "dim": 64, "group": 32, "page": 10,
         "dtype": "f16", "skip": True},
        # one request's step early in its answer: latency is what counts
        {"name": "attend one short", "op": "attend", "batch": 1, "queries": 1, "q_heads": 64, "heads": 8, "dim": 128,
         "group": 64, "page": 64, "length": 500, "ragged": False, "window": 0, "dtype": "bf16", "lse": False},
        # one request with a long context: the work has to be split over the sequence
        {"name": "attend one long", "op": "attend", "batch": 1, "queries": 1, "q_heads": 64, "heads": 8, "dim": 128,
         "group": 64, "page": 64, "length": 131072, "ragged": False, "window": 0, "dtype": "bf16", "lse": False},
        # an ordinary decode batch, sequences of all lengths
        {"name": "attend batch", "op": "attend", "batch": 64, "queries": 1, "q_heads": 64, "heads": 8, "dim": 128,
         "group": 64, "page": 64, "length": 8192, "ragged": True, "window": 0, "dtype": "bf16", "lse": False},
        # fine groups, small pages, four query heads a key head
        {"name": "attend fine groups", "op": "attend", "batch": 32, "queries": 1, "q_heads": 32, "heads": 8, "dim": 128,
         "group": 32, "page": 16, "length": 4001, "ragged": True, "window": 0, "dtype": "f16", "lse": False},
        # four drafted tokens of each request verified at once
        {"name": "attend verify", "op": "attend", "batch": 16, "queries": 4, "q_heads": 64, "heads": 8, "dim": 128,
         "group": 128, "page": 64, "length": 6000, "ragged": True, "window": 0, "dtype": "bf16", "lse": True},
        # every query head has its own keys; pages that end inside a tile
        {"name": "attend own keys", "op": "attend", "batch": 24, "queries": 1, "q_heads": 32, "heads": 32, "dim": 64,
         "group": 64, "page": 100, "length": 2047, "ragged": True, "window": 0, "dtype": "bf16", "lse": False},
        # wide heads that see a window only
        {"name": "attend window", "op": "attend", "batch": 24, "queries": 1, "q_heads": 16, "heads": 4, "dim": 256,
         "group": 128, "page": 32, "length": 20000, "ragged": True, "window": 4096, "dtype": "f16", "lse": True},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend"])
    dim = rng.choice([64, 128, 128, 192, 256])
    group = rng.choice([g for g in (32, 64, 128) if dim % g == 0])
    case = {"op": op, "heads": _log(rng, 1, 32), "dim": dim, "group": group,
            "page": rng.choice([8, 10, 16, 24, 32, 48, 64, 100, 128, 256]), "dtype": rng.choice(["bf16", "f16"])}
    if op != "attend":
        most = 6e7 / (2 * case["heads"] * dim)
        return case | {"tokens": _log(rng, 1, min(65536, int(most))), "skip": rng.random() < 0.3}
    case["batch"] = _log(rng, 1, 256)
    case["queries"] = 1 if rng.random() < 0.6 else rng.randint(2, 8)
    case["q_heads"] = case["heads"] * rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 12, 16])
    case["batch"] = max(1, min(case["batch"], int(4e7) // (case["queries"] * case["q_heads"] * dim)))
    most = min(1.3e8 / (case["batch"] * case["heads"] * dim), 2e9 / (case["batch"] * case["queries"] * case["q_heads"] * dim))
    case["length"] = _log(rng, 1, max(1, min(131072, int(most))))
    return case | {"ragged": rng.random() < 0.6, "window": _log(rng, 1, 8192) if rng.random() < 0.25 else 0,
                   "lse": rng.random() < 0.3}


def _lengths(case):
    """The sequences' lengths: all alike, or spread evenly, the first one a padded request without tokens."""
    n, top = case["batch"], case["length"]
    return [top * i // (n - 1) for i in range(n)] if case["ragged"] and n > 1 else [top] * n


def work(case):
    dim = case["dim"]
    row = dim / 2 + 4 * dim / case["group"]  # codes, scales and offsets of a row of keys or values
    if case["op"] != "attend":
        kept = case["tokens"] * case["heads"] * (0.9 if case["skip"] else 1.0)
        rows = case["tokens"] * case["heads"] * 2
        if case["op"] == "read":
            return {"bytes": 2 * kept * row + rows * 2 * dim + 8 * case["tokens"], "flops": 2 * kept * 2 * dim}
        return {"bytes": 2 * kept * (2 * dim + row) + rows * 2 * dim + 8 * case["tokens"], "flops": 2 * kept * 6 * dim}
    n, window = case["queries"], case["window"]
    read = sum(min(l, window + n - 1) if window else l for l in _lengths(case))
    seen = sum(max(0, min(l - n + i + 1, window or l)) for l in _lengths(case) for i in range(n))
    queries = case["batch"] * n * case["q_heads"]
    return {"bytes": 2 * read * case["heads"] * row + 4 * read / case["page"] + queries * (4 * dim + 4 * case["lse"]),
            "flops": 4 * seen * case["q_heads"] * dim}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _cache(case, g, pages):
    """Codes and (scale, offset) pairs of a cache's keys and values: values of about N(0, 1), keys with offsets of their
    channels."""
    heads, page, dim, groups = case["heads"], case["page"], case["dim"], case["dim"] // case["group"]
    parts = []
    for offset in (1.0, 0.1):
        codes = torch.empty((pages, heads, page, dim // 2), dtype=torch.uint8, device="cuda")
        for part in codes.view(-1, dim // 2).split(1 << 18):
            c = (_randn(g, part.shape[0], dim) * 2.6 - 0.5).round_().clamp_(-8, 7).to(torch.int16)
            part.copy_(((c[:, 0::2] & 15) | ((c[:, 1::2] & 15) << 4)).to(torch.uint8))
        scales = torch.exp(0.2 * _randn(g, pages, heads, page, groups)) / 2.6
        offsets = offset * _randn(g, heads, 1, groups) + 0.2 * _randn(g, pages, heads, page, groups)
        parts += [codes, torch.stack([scales, offsets], dim=-1).to(DTYPES[case["dtype"]])]
    return parts


def prepare(case, seed):
    g = _generator(seed)
    op, dev, dtype = case["op"], "cuda", DTYPES[case["dtype"]]
    heads, page, dim = case["heads"], case["page"], case["dim"]
    st = {"op": op, "group": case["group"], "dtype": dtype}
    if op != "attend":
        tokens = case["tokens"]
        pages = -(-tokens // page) + 2
        # each token's slot, in pages that lie anywhere
        order = torch.randperm(pages, generator=g, device=dev)
        at = torch.arange(tokens, device=dev)
        st["slots"] = order[at // page] * page + at % page
        if case["skip"]:
            st["slots"] = torch.where(torch.rand(tokens, generator=g, device=dev) < 0.1, -1, st["slots"])
        if op == "write":
            bias = _randn(g, heads, dim)
            st["k_in"] = (_randn(g, tokens, heads, dim) + bias).to(dtype)
            x = _randn(g, tokens, heads, dim)
            st["v_in"] = torch.where(torch.rand(x.shape, generator=g, device=dev) < 1e-3, x * 10, x).to(dtype)
            st["cache"] = [torch.zeros((pages, heads, page, *last), dtype=t, device=dev)
                           for _ in range(2) for last, t in (((dim // 2,), torch.uint8), ((dim // case["group"], 2), dtype))]
        else:
            st["cache"] = _cache(case, g, pages)
        st["k"], st["v"] = (torch.empty((tokens, heads, dim), dtype=dtype, device=dev) for _ in range(2))
        return st
    batch, n = case["batch"], case["queries"]
    lengths = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
    lengths = lengths[torch.randperm(batch, generator=g, device=dev)]
    used = (lengths + page - 1) // page
    width = -(-case["length"] // page) + 1  # a table has room for more than the longest sequence
    pages = int(used.sum()) + 3
    order = torch.randperm(pages, generator=g, device=dev).int()
    column = torch.arange(width, device=dev)
    start = torch.cumsum(used, 0) - used
    st["table"] = torch.where(column < used[:, None], order[(start[:, None] + column).clamp(max=pages - 1)], -1).int()
    st["lengths"] = lengths
    st["cache"] = _cache(case, g, pages)
    st["q"] = (1.5 * _randn(g, batch, n, case["q_heads"], dim)).to(dtype)
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty((batch, n, case["q_heads"]), device=dev) if case["lse"] else None
    st["window"] = case["window"]
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    from block_quantized_wire_gb300 import kv4
    if "handle" not in st:  # what a user's program makes once beside its buffers and keeps
        st["handle"] = kv4.Cache(*st["cache"])
        if st["op"] == "attend":
            st["workspace"] = kv4.empty_workspace(st["q"], st["handle"])
    cache = st["handle"]
    if st["op"] == "attend":
        kv4.attend(st["q"], cache, st["table"], st["lengths"], st["out"], st["workspace"], window=st["window"],
                   lse=st["lse"])
        return st["out"] if st["lse"] is None else (st["out"], st["lse"])
    if st["op"] == "write":
        kv4.write(st["k_in"], st["v_in"], st["slots"], cache)
    kv4.read(cache, st["slots"], st["k"], st["v"])
    return st["k"], st["v"]


def _values(codes, scales):
    """The 32-bit values that codes and their (scale, offset) pairs stand for."""
    q = codes.to(torch.int32)
    c = torch.stack([(q << 28) >> 28, (q << 24) >> 28], dim=-1).flatten(-2)
    pairs = scales.float()
    return (c.unflatten(-1, (pairs.shape[-2], -1)) * pairs[..., :1] + pairs[..., 1:]).flatten(-2)


def _quantized(x, group):
    """Packed codes and (scale, offset) pairs of rows."""
    v = x.float().unflatten(-1, (-1, group))
    lo, hi = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
    s = ((hi - lo) / 15).to(x.dtype).float()
    z = ((lo + 4 * s) + 4 * s).to(x.dtype).float()
    c = torch.where(s > 0, ((v - z) / s).round().clamp(-8, 7), 0).flatten(-2).to(torch.int32)
    codes = ((c[..., 0::2] & 15) | ((c[..., 1::2] & 15) << 4)).to(torch.uint8)
    return codes, torch.cat([s, z], dim=-1).to(x.dtype)


def _run_plain(st):
    k, ks, v, vs = st["cache"]
    page = k.shape[2]
    if st["op"] == "attend":
        return _attend_plain(st)
    slots = st["slots"]
    there = slots >= 0
    if st["op"] == "write":
        kept = slots[there]
        codes, pairs = _quantized(st["k_in"][there], st["group"])
        k[kept // page, :, kept % page], ks[kept // page, :, kept % page] = codes, pairs
        codes, pairs = _quantized(st["v_in"][there], st["group"])
        v[kept // page, :, kept % page], vs[kept // page, :, kept % page] = codes, pairs
    at = slots.clamp(min=0)
    where, place = at // page, at % page
    rows = there[:, None, None]
    return (torch.where(rows, _values(k[where, :, place], ks[where, :, place]), 0).to(st["dtype"]),
            torch.where(rows, _values(v[where, :, place], vs[where, :, place]), 0).to(st["dtype"]))


def _attend_plain(st):
    k, ks, v, vs = st["cache"]
    q, table, lengths = st["q"], st["table"].clamp(min=0).long(), st["lengths"].long()
    batch, n, q_heads, dim = q.shape
    heads = k.shape[1]

    def sequence(codes, pairs):  # [batch, heads, positions, dim]
        return _values(codes[table], pairs[table]).transpose(1, 2).flatten(2, 3)

    rows = q.float().unflatten(2, (heads, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [batch, heads, n * shared, dim]
    scores = (rows @ sequence(k, ks).transpose(2, 3)) * dim ** -0.5
    position = torch.arange(scores.shape[-1], device=q.device)
    last = lengths[:, None] - n + torch.arange(n, device=q.device)  # the last position that a query sees
    seen = position <= last[..., None]
    if st["window"]:
        seen &= position > last[..., None] - st["window"]
    seen = seen.repeat_interleave(q_heads // heads, dim=1)[:, None]
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > -math.inf, top, 0))
    total = p.sum(-1, keepdim=True)
    out = (p @ sequence(v, vs)) / torch.where(total > 0, total, 1)

    def by_query(t):
        return t.unflatten(2, (n, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)

    out = by_query(out).to(q.dtype)
    return out if st["lse"] is None else (out, by_query(torch.log(total) + torch.where(total > 0, top, 0))[..., 0])


# ------------------------------------------------------------------ 64 bits
def _wide(codes, scales):
    """Values in 64 bits, from a table of the sixteen codes."""
    table = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1], dtype=torch.float64, device="cuda")
    c = torch.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=torch.float64, device="cuda")
    c[..., 0::2] = table[(codes & 15).long()]
    c[..., 1::2] = table[(codes >> 4).long()]
    group = c.shape[-1] // scales.shape[-2]
    wide = scales.to(torch.float64).repeat_interleave(group, dim=-2)
    return c * wide[..., 0] + wide[..., 1]


def _round_trip(x, group):
    """A row as the cache gives it back: the scale and the offset are rounded to the rows' type, the difference from the
    offset to 32 bits, as the definition has it; the rest is exact in 64 bits."""
    v = x.to(torch.float64).unflatten(-1, (-1, group))
    lo, hi = v.min(-1, keepdim=True).values, v.max(-1, keepdim=True).values
    s = ((hi.float() - lo.float()) / 15).to(x.dtype).to(torch.float64)
    z = ((lo.float() + 4 * s.float()) + 4 * s.float()).to(x.dtype).to(torch.float64)
    code = torch.round((v - z).float().to(torch.float64) / torch.where(s > 0, s, 1))
    return (torch.where(s > 0, code.clamp(-8, 7), 0) * s + z).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    k, ks, v, vs = st["cache"]
    page = case["page"]
    if st["op"] != "attend":
        outs = []
        for codes, pairs, rows in ((k, ks, st.get("k_in")), (v, vs, st.get("v_in"))):
            parts = []
            for lo in range(0, case["tokens"], 4096):
                slots = st["slots"][lo:lo + 4096]
                at = slots.clamp(min=0)
                part = _round_trip(rows[lo:lo + 4096], case["group"]) if rows is not None else \
                    _wide(codes[at // page, :, at % page], pairs[at // page, :, at % page])
                parts.append(part * (slots >= 0)[:, None, None])
            outs.append(torch.cat(parts))
        return tuple(outs)
    q, n, heads = st["q"], case["queries"], case["heads"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    for b, length in enumerate(st["lengths"].tolist()):
        pages = st["table"][b, :-(-length // page)].long()
        for h in range(heads if length else 0):
            keys = _wide(k[pages, h], ks[pages, h]).flatten(0, 1)[:length]
            values = _wide(v[pages, h], vs[pages, h]).flatten(0, 1)[:length]
            shared = slice(h * case["q_heads"] // heads, (h + 1) * case["q_heads"] // heads)
            for i in range(n):
                hi = length - n + i + 1
                lo = max(0, hi - case["window"]) if case["window"] else 0
                if hi > lo:
                    x = (q[b, i, shared].to(torch.float64) @ keys[lo:hi].T) / math.sqrt(case["dim"])
                    lse[b, i, shared] = torch.logsumexp(x, dim=1)
                    out[b, i, shared] = torch.softmax(x, dim=1) @ values[lo:hi]
    return (out, lse) if case["lse"] else out
