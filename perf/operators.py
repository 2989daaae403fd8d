"""The expert-layer operators as measured: their cases, inputs, plain forms and exact values.

One mixture-of-experts layer, as a serving or training program runs it around the codec's all-reduce payloads:

* ``sort``          expert ids of the router -> the tokens' places grouped by expert
* ``gather``        token rows copied to their places (``gather_grad``: back, summed per token)
* ``combine``       expert rows brought back, weighted and summed per token (``combine_grad``: its gradients)
* ``matvec``        a few rows times a 4-bit weight matrix with group scales
* ``experts``       the same product with each sorted row's own expert

``run`` computes them with elementary torch operations in 32 bits (``own`` false) or with this repository's kernels
(``own`` true). ``exact`` restates the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "i32": 4, "i64": 8}
SORT_PARTS = 128  # rows of the sort's workspace


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 16 requests: the router's top-8 of 256 experts, as torch.topk returns it
        {"name": "sort decode", "op": "sort", "tokens": 16, "k": 8, "experts": 256, "total": 256, "ids": "i64"},
        # a whole prefill batch on a GPU that holds a quarter of the experts
        {"name": "sort prefill", "op": "sort", "tokens": 65536, "k": 8, "experts": 64, "total": 256, "ids": "i32"},
        # dispatch of a prefill batch at the projection width of the codec's workloads
        {"name": "gather prefill", "op": "gather", "tokens": 16384, "k": 8, "experts": 256, "total": 256,
         "hidden": 7168, "dtype": "bf16"},
        # the dispatch's gradient in a small training step, an odd width that no vector access fits
        {"name": "gather grad odd", "op": "gather_grad", "tokens": 1999, "k": 6, "experts": 40, "total": 60,
         "hidden": 1001, "dtype": "f16"},
        # the decode step's way back: latency is what counts
        {"name": "combine decode", "op": "combine", "tokens": 16, "k": 8, "experts": 256, "total": 256,
         "hidden": 7168, "dtype": "bf16"},
        # the prefill batch's way back, with half of the experts held here
        {"name": "combine prefill", "op": "combine", "tokens": 16384, "k": 8, "experts": 128, "total": 256,
         "hidden": 7168, "dtype": "bf16"},
        # a training step's way back through the layer
        {"name": "combine grad train", "op": "combine_grad", "tokens": 8192, "k": 8, "experts": 64, "total": 64,
         "hidden": 4096, "dtype": "bf16"},
        # the same in 32 bits with two experts a token
        {"name": "combine grad f32", "op": "combine_grad", "tokens": 3000, "k": 2, "experts": 8, "total": 8,
         "hidden": 1028, "dtype": "f32"},
        # a projection of one decoding request
        {"name": "matvec one token", "op": "matvec", "rows": 1, "n": 7168, "inner": 7168, "group": 128,
         "dtype": "bf16", "scales": "bf16"},
        # a wide projection of a small decode batch, fine groups
        {"name": "matvec 16 tokens", "op": "matvec", "rows": 16, "n": 18432, "inner": 7168, "group": 32,
         "dtype": "f16", "scales": "f16"},
        # the gate and up products of one token's eight experts
        {"name": "experts one token", "op": "experts", "tokens": 1, "k": 8, "experts": 64, "total": 64, "n": 4096,
         "inner": 7168, "group": 32, "dtype": "bf16", "scales": "bf16", "sorted": False},
        # the down products of a decode batch, an odd output width, rows already sorted
        {"name": "experts decode batch", "op": "experts", "tokens": 24, "k": 6, "experts": 48, "total": 64,
         "n": 7000, "inner": 2048, "group": 64, "dtype": "bf16", "scales": "f32", "sorted": True},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sort", "gather", "gather_grad", "combine", "combine_grad", "matvec", "experts"])
    if op == "matvec":
        group = rng.choice([32, 64, 128])
        dtype = rng.choice(["bf16", "f16"])
        return {"op": op, "rows": _log(rng, 1, 32), "n": _log(rng, 500, 20000),
                "inner": group * _log(rng, 1024 // group, 16384 // group), "group": group, "dtype": dtype,
                "scales": rng.choice([dtype, "f32"])}
    total = _log(rng, 8, 256)
    k = min(_log(rng, 1, 16), total)
    experts = total if rng.random() < 0.5 else max(1, total // rng.choice([2, 3, 4]))
    if op == "sort":
        return {"op": op, "tokens": _log(rng, 1, 65536), "k": min(k, 8), "experts": experts, "total": total,
                "ids": rng.choice(["i32", "i64"])}
    if op == "experts":
        group = rng.choice([32, 64, 128])
        dtype = rng.choice(["bf16", "f16"])
        total = min(total, 64)
        k = min(k, 8, total)
        return {"op": op, "tokens": _log(rng, 1, 32), "k": k, "experts": min(experts, total), "total": total,
                "n": _log(rng, 500, 4500), "inner": group * _log(rng, 512 // group, 6144 // group), "group": group,
                "dtype": dtype, "scales": rng.choice([dtype, "f32"]), "sorted": rng.random() < 0.5}
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    hidden = _log(rng, 256, 7168)
    if rng.random() < 0.7:
        hidden = 8 * (hidden // 8)
    most = 1.2e9 / (2 * hidden * k * SIZE[dtype])
    return {"op": op, "tokens": _log(rng, 1, max(1, min(16384, int(most)))), "k": k, "experts": experts,
            "total": total, "hidden": hidden, "dtype": dtype}


def work(case):
    op = case["op"]
    if op == "matvec":
        m, n, inner = case["rows"], case["n"], case["inner"]
        weights = n * inner / 2 + n * (inner // case["group"]) * SIZE[case["scales"]]
        return {"bytes": weights + 2 * m * (inner + n), "flops": 2 * m * n * inner}
    t, k = case["tokens"], case["k"]
    slots, kept = t * k, t * k * case["experts"] / case["total"]
    if op == "sort":
        return {"bytes": slots * (SIZE[case["ids"]] + 8) + 4 * (case["experts"] + 1), "flops": 0}
    if op == "experts":
        n, inner = case["n"], case["inner"]
        active = case["experts"] * (1 - (1 - k / case["total"]) ** t)  # experts that a batch reaches, on average
        weights = active * (n * inner / 2 + n * (inner // case["group"]) * SIZE[case["scales"]])
        return {"bytes": weights + 2 * (kept if case["sorted"] else t) * inner + 2 * slots * n,
                "flops": 2 * kept * n * inner}
    row = case["hidden"] * SIZE[case["dtype"]]
    if op == "gather":
        return {"bytes": (t + slots) * row + 4 * slots, "flops": 0}
    if op == "gather_grad":
        return {"bytes": (t + kept) * row + 4 * slots, "flops": kept * case["hidden"]}
    if op == "combine":
        return {"bytes": (t + kept) * row + 8 * slots, "flops": 2 * kept * case["hidden"]}
    return {"bytes": (t + kept + slots) * row + 12 * slots, "flops": 3 * kept * case["hidden"]}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, *shape):
    """N(0, 1) with one value in a thousand twenty times as large, as activations have them."""
    x = _randn(g, *shape)
    return torch.where(torch.rand(shape, generator=g, device="cuda") < 1e-3, x * 20, x)


def _route(case, g):
    """The router's choice: k different experts of `total` for each token, some more popular than others, as ids of the
    experts held here (others lie outside [0, experts)), and weights that sum to 1."""
    scores = _randn(g, case["tokens"], case["total"]) + 0.5 * _randn(g, case["total"])
    top, ids = scores.topk(case["k"], dim=1)
    return ids - (case["total"] - case["experts"]) // 2, torch.softmax(top, dim=1)


def _sorted(ids, n_experts):
    """offsets, order and inverse of the stable sort by expert."""
    flat = ids.reshape(-1)
    here = (flat >= 0) & (flat < n_experts)
    key = torch.where(here, flat, n_experts)
    by = torch.argsort(key, stable=True)
    place = torch.empty_like(by)
    at = torch.arange(flat.numel(), device=flat.device)
    place[by] = at
    ends = torch.cumsum((key[None, :] == torch.arange(n_experts, device=flat.device)[:, None]).sum(1), 0) \
        if flat.numel() * n_experts < 1 << 22 else torch.cumsum(torch.bincount(key, minlength=n_experts + 1)[:n_experts], 0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    order = torch.where(at < offsets[-1], by, -1)
    inverse = torch.where(here, place, -1)
    return offsets.int(), order.int(), inverse.int().view(ids.shape)


def _weights(case, g, *lead):
    """4-bit codes of a normal distribution and their group scales: two codes a byte, the lower column in the low half."""
    n, inner, group = case["n"], case["inner"], case["group"]
    q = torch.empty((*lead, n, inner // 2), dtype=torch.uint8, device="cuda")
    for part in q.view(-1, n, inner // 2):
        c = (_randn(g, n, inner) * 2.4).round_().clamp_(-7, 7).to(torch.int16)
        part.copy_(((c[:, 0::2] & 15) | ((c[:, 1::2] & 15) << 4)).to(torch.uint8))
    s = torch.exp(0.3 * _randn(g, *lead, n, inner // group)) * (0.02 / 2.4)
    return q, s.to(DTYPES[case["scales"]])


def prepare(case, seed):
    g = _generator(seed)
    op, dev = case["op"], "cuda"
    st = {"op": op, "group": case.get("group")}
    if op == "matvec":
        st["x"] = _activations(g, case["rows"], case["inner"]).to(DTYPES[case["dtype"]])
        st["q"], st["s"] = _weights(case, g)
        st["out"] = torch.empty((case["rows"], case["n"]), dtype=st["x"].dtype, device=dev)
        return st
    t, k, n_experts = case["tokens"], case["k"], case["experts"]
    ids, weights = _route(case, g)
    st |= {"k": k, "experts": n_experts}
    if op == "sort":
        st["ids"] = ids.int() if case["ids"] == "i32" else ids
        st["offsets"] = torch.empty(n_experts + 1, dtype=torch.int32, device=dev)
        st["order"] = torch.empty(t * k, dtype=torch.int32, device=dev)
        st["inverse"] = torch.empty((t, k), dtype=torch.int32, device=dev)
        st["workspace"] = torch.empty((SORT_PARTS, n_experts), dtype=torch.int32, device=dev)
        return st
    st["offsets"], st["order"], st["inverse"] = _sorted(ids, n_experts)
    if op == "experts":
        rows = t * k if case["sorted"] else t
        st["x"] = _activations(g, rows, case["inner"]).to(DTYPES[case["dtype"]])
        st["sorted"] = case["sorted"]
        st["q"], st["s"] = _weights(case, g, n_experts)
        st["out"] = torch.empty((t * k, case["n"]), dtype=st["x"].dtype, device=dev)
        return st
    dtype, hidden = DTYPES[case["dtype"]], case["hidden"]
    st["weights"] = weights
    if op in ("gather", "combine_grad"):
        st["x"] = _activations(g, t, hidden).to(dtype)  # the tokens, or the gradient of the layer's output
    if op != "gather":
        st["y"] = _activations(g, t * k, hidden).to(dtype)  # rows by expert
    if op in ("gather", "combine_grad"):
        st["out"] = torch.empty((t * k, hidden), dtype=dtype, device=dev)
    else:
        st["out"] = torch.empty((t, hidden), dtype=dtype, device=dev)
    if op == "combine_grad":
        st["dweights"] = torch.empty((t, k), dtype=torch.float32, device=dev)
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    from block_quantized_wire_gb300 import experts, w4
    op = st["op"]
    if op == "matvec":
        w4.matvec_w4(st["x"], st["q"], st["s"], st["out"])
        return st["out"]
    if op == "experts":
        w4.matvec_w4_experts(st["x"], st["q"], st["s"], st["offsets"], st["out"],
                             order=None if st["sorted"] else st["order"], top_k=st["k"])
        return st["out"]
    if op == "sort":
        experts.sort(st["ids"], st["experts"], st["offsets"], st["order"], st["inverse"], st["workspace"])
        return st["offsets"], st["order"], st["inverse"]
    if op == "gather":
        experts.gather(st["x"], st["inverse"], st["offsets"], st["out"])
        return st["out"]
    if op == "gather_grad":
        experts.gather_grad(st["y"], st["inverse"], st["out"])
        return st["out"]
    if op == "combine":
        experts.combine(st["y"], st["weights"], st["inverse"], st["out"])
        return st["out"]
    experts.combine_grad(st["x"], st["y"], st["weights"], st["inverse"], st["offsets"], st["out"], st["dweights"])
    return st["out"], st["dweights"]


def _dequantized(q, s, group, dtype):
    """The weights that codes and scales stand for: [..., n, inner]."""
    q = q.to(torch.int32)
    c = torch.stack([(q << 28) >> 28, (q << 24) >> 28], dim=-1).flatten(-2)
    return (c.unflatten(-1, (-1, group)).to(dtype) * s.to(dtype)[..., None]).flatten(-2)


def _run_plain(st):
    op = st["op"]
    if op == "matvec":
        w = _dequantized(st["q"], st["s"], st["group"], torch.float32)
        return (st["x"].float() @ w.T).to(st["x"].dtype)
    if op == "sort":
        return _sorted(st["ids"], st["experts"])
    order, inverse = st["order"].long(), st["inverse"].long()
    kept, here = order >= 0, inverse >= 0
    token = order.clamp(min=0) // st["k"]
    if op == "experts":
        x, offsets = st["x"], st["offsets"].long()
        counts = offsets[1:] - offsets[:-1]
        used = torch.nonzero(counts).flatten()
        w = _dequantized(st["q"][used], st["s"][used], st["group"], torch.float32)
        rows = x.float() if st["sorted"] else x.float()[token]
        at = torch.arange(order.numel(), device=x.device)
        expert = torch.bucketize(at, offsets[1:], right=True).clamp(max=counts.numel() - 1)
        slot = (torch.cumsum(counts > 0, 0) - 1)[expert]
        nth = at - offsets[expert]
        where = torch.nonzero(kept).flatten()
        padded = torch.zeros((used.numel(), int(counts.max()), x.shape[1]), device=x.device)
        padded[slot[where], nth[where]] = rows[where]
        y = torch.bmm(padded, w.transpose(1, 2))
        out = torch.zeros((order.numel(), w.shape[1]), device=x.device)
        out[where] = y[slot[where], nth[where]]
        return out.to(x.dtype)
    if op == "gather":
        return torch.where(kept[:, None], st["x"][token], 0)
    y = st["y"]
    rows = torch.where(here[..., None], y[inverse.clamp(min=0)].float(), 0)
    if op == "gather_grad":
        return rows.sum(1).to(y.dtype)
    if op == "combine":
        return (rows * st["weights"][..., None]).sum(1).to(y.dtype)
    dout = st["x"].float()
    weight = st["weights"].reshape(-1)[order.clamp(min=0)]
    dy = torch.where(kept[:, None], weight[:, None] * dout[token], 0).to(y.dtype)
    return dy, (rows * dout[:, None, :]).sum(2)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op, f64 = st["op"], torch.float64
    if op == "sort":
        return None
    if op == "matvec":
        return torch.cat([st["x"].to(f64) @ _w64(q, s, st["group"]).T
                          for q, s in zip(st["q"].split(4096), st["s"].split(4096))], dim=1)
    k, inverse = st["k"], st["inverse"].long()
    if op == "gather":
        out = torch.zeros(st["out"].shape, dtype=f64, device="cuda")
        for t in range(0, inverse.shape[0], 1024):
            places = inverse[t:t + 1024]
            here = places >= 0
            out[places[here]] = st["x"][t:t + 1024].to(f64).repeat_interleave(here.sum(1), dim=0)
        return out
    if op == "experts":
        out = torch.zeros(st["out"].shape, dtype=f64, device="cuda")
        ends = st["offsets"].tolist()
        for e in range(st["experts"]):
            lo, hi = ends[e], ends[e + 1]
            if lo < hi:
                at = slice(lo, hi) if st["sorted"] else st["order"][lo:hi].long() // k
                out[lo:hi] = st["x"][at].to(f64) @ _w64(st["q"][e], st["s"][e], st["group"]).T
        return out
    y, weights = st["y"], st["weights"].to(f64)
    if op == "combine_grad":
        dy = torch.zeros(y.shape, dtype=f64, device="cuda")
        dw = torch.zeros(weights.shape, dtype=f64, device="cuda")
    out = torch.zeros((inverse.shape[0], y.shape[1]), dtype=f64, device="cuda")
    for j in range(k):
        t = torch.nonzero(inverse[:, j] >= 0).flatten()
        p = inverse[t, j]
        if op == "gather_grad":
            out[t] += y[p].to(f64)
        elif op == "combine":
            out[t] += weights[t, j, None] * y[p].to(f64)
        else:
            dout = st["x"][t].to(f64)
            dy[p] = weights[t, j, None] * dout
            dw[t, j] = (dout * y[p].to(f64)).sum(1)
    return (dy, dw) if op == "combine_grad" else out


def _w64(q, s, group):
    """Codes and scales in 64 bits, from a table of the sixteen codes."""
    table = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1], dtype=torch.float64, device=q.device)
    w = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device=q.device)
    w[:, 0::2] = table[(q & 15).long()]
    w[:, 1::2] = table[(q >> 4).long()]
    return w * s.to(torch.float64).repeat_interleave(group, dim=1)
