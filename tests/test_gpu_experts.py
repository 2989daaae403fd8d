"""The expert layer's token kernels (sort, gather, combine and their gradients) against
plain 64-bit restatements of their definitions.

Tolerances. A sum of n products in binary32, one fused multiply-add each, is off by at
most n * 2^-24 * sum |terms| (to first order; the factor 1.01 covers the rest), and one
rounding to the row type adds 2^-p * |result| (p = 8 for BF16, 11 for FP16, 24 for FP32)
or half the type's smallest subnormal. Places, copies and zeros are compared bit for bit.
"""
import numpy as np
import pytest
import torch

from block_quantized_wire_gb300 import _lib, build, codec, experts
from tests.helpers import Guarded

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (torch.bfloat16, 8, 2.0 ** -134), "f16": (torch.float16, 11, 2.0 ** -25),
         "f32": (torch.float32, 24, 2.0 ** -150)}


def ids_of(rng, tokens, top_k, n_experts, drop=0.2, skew=False):
    """Choices, some of them held elsewhere (below 0 or at n_experts and above)."""
    ids = rng.integers(0, n_experts, (tokens, top_k))
    if skew:
        ids = np.minimum(ids, rng.integers(0, n_experts, (tokens, top_k)) // 4)
    away = rng.random((tokens, top_k)) < drop
    return np.where(away, rng.choice([-1, -7, n_experts, n_experts + 3], (tokens, top_k)), ids)


def plan_of(ids, n_experts):
    """offsets, order, inverse by the definition."""
    flat = ids.reshape(-1)
    order, offsets = [], [0]
    by = np.argsort(np.where((flat >= 0) & (flat < n_experts), flat, n_experts), kind="stable")
    kept = int(((flat >= 0) & (flat < n_experts)).sum())
    order = np.full(flat.size, -1, np.int32)
    order[:kept] = by[:kept]
    inverse = np.full(flat.size, -1, np.int32)
    inverse[by[:kept]] = np.arange(kept)
    offsets = np.searchsorted(flat[by[:kept]], np.arange(n_experts + 1)).astype(np.int32)
    return offsets, order, inverse.reshape(ids.shape)


def device_plan(ids, n_experts):
    return [torch.from_numpy(a).cuda() for a in plan_of(ids, n_experts)]


def rows_in(rng, rows, cols, dtype, ld=None, offset=0):
    """A [rows, cols] view with leading dimension ld whose first value is `offset` values
    past a 256-byte boundary."""
    ld = cols if ld is None else ld
    base = torch.from_numpy(rng.standard_normal(offset + max(rows, 1) * ld).astype(np.float32)).to(dtype).cuda()
    return torch.as_strided(base, (rows, cols), (ld, 1), offset)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def check_close(got, want, terms, n, p, tiny):
    """|got - want| within the bound above; `terms` is sum |terms| of each value's sum."""
    bound = 1.01 * (n * 2.0 ** -24 * terms + 2.0 ** -p * np.abs(want)) + tiny
    err = np.abs(f64(got) - want)
    assert np.all(err <= bound), float((err - bound).max())


# ------------------------------------------------------------------ sort
SORTS = [(1, 1, 1), (1, 8, 256), (16, 8, 256), (3, 5, 7), (513, 8, 64), (1365, 3, 1024), (1366, 3, 1023),
         (4097, 1, 2), (5000, 7, 96), (20000, 16, 384), (65536, 8, 64)]


@pytest.mark.parametrize("tokens,top_k,n_experts", SORTS)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort_is_the_stable_order_by_expert(tokens, top_k, n_experts, dtype):
    rng = np.random.default_rng(tokens + top_k)
    ids = ids_of(rng, tokens, top_k, n_experts, drop=0.25, skew=tokens % 2 == 0)
    want = plan_of(ids, n_experts)
    slots = tokens * top_k
    bufs = [Guarded(4 * n) for n in (n_experts + 1, slots, slots, experts.SORT_PARTS * n_experts)]
    offsets, order, inverse, ws = (b.view(torch.int32) for b in bufs)
    inverse = inverse.view(tokens, top_k)
    experts.sort(torch.from_numpy(ids).to(dtype).cuda(), n_experts, offsets, order, inverse, ws)
    for got, ref in zip((offsets, order, inverse), want):
        assert np.array_equal(got.cpu().numpy(), ref)
    assert all(b.bands_intact() for b in bufs)


@pytest.mark.parametrize("tokens", [0, 1, 9, 3000])
@pytest.mark.parametrize("fill", [-1, 64, 2 ** 40, -2 ** 40])
def test_sort_with_no_slot_kept(tokens, fill):
    # 2^40 has the low 32 bits of expert 0: an id is compared whole
    plan = experts.empty_plan(tokens, 4, 64)
    experts.sort(torch.full((tokens, 4), fill, dtype=torch.int64, device="cuda"), 64, *plan)
    assert not plan.offsets.any() and bool((plan.order == -1).all()) and bool((plan.inverse == -1).all())


@pytest.mark.parametrize("tokens", [40, 4000])
def test_sort_with_one_expert_taking_all(tokens):
    plan = experts.empty_plan(tokens, 4, 300)
    experts.sort(torch.full((tokens, 4), 299, dtype=torch.int32, device="cuda"), 300, *plan)
    n = tokens * 4
    assert plan.offsets[299].item() == 0 and plan.offsets[300].item() == n
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    assert torch.equal(plan.order, at) and torch.equal(plan.inverse.reshape(-1), at)


# ------------------------------------------------------------------ gather, combine, gradients
# tokens, top_k, hidden, leading dimension minus hidden, offset of the first value
SHAPES = [(1, 1, 1, 0, 0), (1, 8, 7168, 0, 0), (5, 3, 129, 0, 0), (7, 2, 8, 8, 0), (33, 6, 1001, 0, 0),
          (9, 4, 512, 3, 0), (17, 16, 320, 0, 1), (64, 8, 2048, 64, 8), (3, 40, 96, 0, 0), (1030, 2, 24, 0, 0),
          (12, 5, 4104, 0, 0)]


def setup(name, tokens, top_k, hidden, pad, offset, drop=0.3):
    dtype, p, tiny = TYPES[name]
    rng = np.random.default_rng(tokens * 1000 + hidden)
    n_experts = 11
    ids = ids_of(rng, tokens, top_k, n_experts, drop)
    offsets, order, inverse = plan_of(ids, n_experts)
    return dtype, p, tiny, rng, hidden + pad, offset, offsets, order, inverse


def guarded_rows(rows, cols, ld, offset, dtype):
    """A guarded [rows, cols] view like rows_in's, filled with the sentinel, and its guard."""
    size = torch.empty((), dtype=dtype).element_size()
    g = Guarded(size * (offset + rows * ld))
    return g.view(dtype)[offset:].view(rows, ld)[:, :cols], g


def untouched_between(g, view, ld, offset):
    """True if nothing but the view's own values was written."""
    rows, cols = view.shape
    raw, fresh = g.view(view.dtype).clone(), Guarded(g.nbytes).view(view.dtype)
    for t in (raw, fresh):
        t[offset:].view(rows, ld)[:, :cols] = 0
    return g.bands_intact() and torch.equal(raw.view(torch.uint8), fresh.view(torch.uint8))


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_gather_copies_rows_to_their_places(name, shape):
    tokens, top_k, hidden, pad, off = shape
    dtype, _, _, rng, ld, offset, offsets, order, inverse = setup(name, *shape)
    x = rows_in(rng, tokens, hidden, dtype, ld, offset)
    x[0, 0] = float("nan")
    out, g = guarded_rows(tokens * top_k, hidden, ld, offset, dtype)
    experts.gather(x, torch.from_numpy(inverse).cuda(), torch.from_numpy(offsets).cuda(), out)
    want = torch.zeros_like(out)
    kept = torch.from_numpy(order[order >= 0]).cuda().long()
    want[:kept.numel()] = x[kept // top_k]
    size = want.element_size()
    assert torch.equal(out.contiguous().view(torch.int16 if size == 2 else torch.int32),
                       want.view(torch.int16 if size == 2 else torch.int32))
    assert untouched_between(g, out, ld, offset)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_combine_sums_a_tokens_rows(name, shape, weighted):
    tokens, top_k, hidden, pad, off = shape
    dtype, p, tiny, rng, ld, offset, offsets, order, inverse = setup(name, *shape)
    y = rows_in(rng, tokens * top_k, hidden, dtype, ld, offset)
    weights = rng.standard_normal((tokens, top_k)).astype(np.float32)
    kept = int(offsets[-1])
    y[kept:] = float("nan")            # rows at places that no slot takes
    given = np.where(inverse >= 0, weights, np.float32("nan"))  # dropped slots' weights
    out, g = guarded_rows(tokens, hidden, ld, offset, dtype)
    inv = torch.from_numpy(inverse).cuda()
    if weighted:
        experts.combine(y, torch.from_numpy(given).cuda(), inv, out)
    else:
        experts.gather_grad(y, inv, out)
        weights = np.ones_like(weights)
    y64 = f64(y)
    want, terms = np.zeros((tokens, hidden)), np.zeros((tokens, hidden))
    for j in range(top_k):
        t = np.nonzero(inverse[:, j] >= 0)[0]
        term = weights[t, j, None].astype(np.float64) * y64[inverse[t, j]]
        want[t] += term
        terms[t] += np.abs(term)
    check_close(out, want, terms, top_k, p, tiny)
    assert untouched_between(g, out, ld, offset)


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_combine_grad_against_the_formula(name, shape):
    tokens, top_k, hidden, pad, off = shape
    dtype, p, tiny, rng, ld, offset, offsets, order, inverse = setup(name, *shape)
    dout = rows_in(rng, tokens, hidden, dtype, ld, offset)
    y = rows_in(rng, tokens * top_k, hidden, dtype, ld, offset)
    kept = int(offsets[-1])
    y[kept:] = float("nan")
    weights = np.where(inverse >= 0, rng.standard_normal((tokens, top_k)), np.nan).astype(np.float32)
    dy, g = guarded_rows(tokens * top_k, hidden, ld, offset, dtype)
    gw = Guarded(4 * tokens * top_k)
    dw = gw.view(torch.float32, (tokens, top_k))
    experts.combine_grad(dout, y, torch.from_numpy(weights).cuda(), torch.from_numpy(inverse).cuda(),
                         torch.from_numpy(offsets).cuda(), dy, dw)
    d64, y64 = f64(dout), f64(y)
    slot = order[:kept]
    want_dy = np.zeros((tokens * top_k, hidden))
    want_dy[:kept] = weights.reshape(-1)[slot, None].astype(np.float64) * d64[slot // top_k]
    check_close(dy, want_dy, np.abs(want_dy), 1, p, tiny)
    assert not dy[kept:].any()
    want_dw, terms = np.zeros(tokens * top_k), np.zeros(tokens * top_k)
    want_dw[slot] = (d64[slot // top_k] * y64[:kept]).sum(1)
    terms[slot] = np.abs(d64[slot // top_k] * y64[:kept]).sum(1)
    check_close(dw.reshape(-1), want_dw, terms, hidden, 24, 0.0)
    assert untouched_between(g, dy, ld, offset) and gw.bands_intact()


def test_combine_grad_against_differences():
    # combine is linear in y and in the weights, so a central difference with step 1 is the
    # derivative up to the forward's rounding: each output is off by at most
    # (top_k + 1) * 2^-24 * sum |terms|, and the loss adds up hidden of them
    rng = np.random.default_rng(5)
    tokens, top_k, hidden, n_experts = 6, 3, 40, 4
    ids = ids_of(rng, tokens, top_k, n_experts)
    offsets, order, inverse = device_plan(ids, n_experts)
    y = rows_in(rng, tokens * top_k, hidden, torch.float32)
    dout = rows_in(rng, tokens, hidden, torch.float32)
    w = torch.from_numpy(rng.standard_normal((tokens, top_k)).astype(np.float32)).cuda()
    dy, dw = torch.empty_like(y), torch.empty_like(w)
    experts.combine_grad(dout, y, w, inverse, offsets, dy, dw)
    out = torch.empty((tokens, hidden), device="cuda")

    def loss(y, w):
        experts.combine(y, w, inverse, out)
        return float((out.double() * dout.double()).sum())

    biggest = float(dout.abs().max()) * (top_k + 1) * (float(y.abs().max()) + 1) * (float(w.abs().max()) + 1)
    tol = 2 * tokens * hidden * (top_k + 1) * 2.0 ** -24 * biggest
    for t in range(tokens):
        for j in range(top_k):
            up, down = w.clone(), w.clone()
            up[t, j] += 1.0
            down[t, j] -= 1.0
            assert abs((loss(y, up) - loss(y, down)) / 2 - float(dw[t, j])) <= tol
    for p in range(0, tokens * top_k, 4):
        for c in (0, 17, 39):
            up, down = y.clone(), y.clone()
            up[p, c] += 1.0
            down[p, c] -= 1.0
            assert abs((loss(up, w) - loss(down, w)) / 2 - float(dy[p, c])) <= tol


def test_gather_grad_against_differences():
    rng = np.random.default_rng(6)
    tokens, top_k, hidden, n_experts = 5, 4, 33, 3
    offsets, order, inverse = device_plan(ids_of(rng, tokens, top_k, n_experts), n_experts)
    x = rows_in(rng, tokens, hidden, torch.float32)
    dout = rows_in(rng, tokens * top_k, hidden, torch.float32)
    dx = torch.empty_like(x)
    experts.gather_grad(dout, inverse, dx)
    out = torch.empty_like(dout)

    def loss(x):
        experts.gather(x, inverse, offsets, out)
        return float((out.double() * dout.double()).sum())

    tol = 4 * 2.0 ** -24 * top_k * float(dout.abs().max()) * 4  # x +- 1 is rounded, and dx's sum
    for t in range(tokens):
        for c in range(0, hidden, 8):
            up, down = x.clone(), x.clone()
            up[t, c] += 1.0
            down[t, c] -= 1.0
            assert abs((loss(up) - loss(down)) / 2 - float(dx[t, c])) <= tol


def test_infinities_and_nan_stay_with_their_token():
    rng = np.random.default_rng(8)
    tokens, top_k, hidden, n_experts = 6, 2, 64, 5
    ids = ids_of(rng, tokens, top_k, n_experts, drop=0.0)
    offsets, order, inverse = device_plan(ids, n_experts)
    y = rows_in(rng, tokens * top_k, hidden, torch.bfloat16)
    w = torch.ones((tokens, top_k), device="cuda")
    out, clean = torch.empty((tokens, hidden), dtype=torch.bfloat16, device="cuda"), None
    clean = torch.empty_like(out)
    experts.combine(y, w, inverse, clean)
    y[inverse[2, 1].item(), 5] = float("inf")
    y[inverse[4, 0].item(), 6] = float("nan")
    experts.combine(y, w, inverse, out)
    assert out[2, 5].item() == float("inf") and bool(out[4, 6].isnan())
    out[2, 5], out[4, 6] = clean[2, 5], clean[4, 6]
    assert torch.equal(out, clean)


def test_empty_batches_and_columns():
    e = torch.empty
    inv0 = e((0, 4), dtype=torch.int32, device="cuda")
    offsets = torch.zeros(6, dtype=torch.int32, device="cuda")
    none = e((0, 16), device="cuda")
    experts.gather(none, inv0, offsets, none)
    experts.combine(none, e((0, 4), device="cuda"), inv0, none)
    experts.combine_grad(none, none, e((0, 4), device="cuda"), inv0, offsets, none, e((0, 4), device="cuda"))
    offsets, order, inverse = device_plan(np.array([[0, 1], [1, 9]]), 5)
    thin = e((2, 0), device="cuda")
    experts.gather(thin, inverse, offsets, e((4, 0), device="cuda"))
    experts.combine(e((4, 0), device="cuda"), None, inverse, thin)
    dw = torch.full((2, 2), 7.0, device="cuda")
    experts.combine_grad(thin, e((4, 0), device="cuda"), torch.ones((2, 2), device="cuda"), inverse, offsets,
                         e((4, 0), device="cuda"), dw)
    assert not dw.any()


def test_offsets_past_2_31_values():
    # places whose first value lies past 2^31 values (and 2^32 bytes) of the buffer
    tokens, top_k, hidden = 70000, 8, 4096
    ids = torch.arange(tokens * top_k, device="cuda", dtype=torch.int32).view(tokens, top_k) % 16
    plan = experts.empty_plan(tokens, top_k, 16)
    experts.sort(ids, 16, *plan)
    x = torch.randn((tokens, hidden), device="cuda", dtype=torch.bfloat16)
    out = torch.empty((tokens * top_k, hidden), device="cuda", dtype=torch.bfloat16)
    experts.gather(x, plan.inverse, plan.offsets, out)
    last = tokens * top_k - 5
    assert torch.equal(out[last:], x[(plan.order[last:] // top_k).long()])
    back = torch.empty_like(x)
    experts.combine(out, torch.full((tokens, top_k), 0.125, device="cuda"), plan.inverse, back)
    assert torch.equal(back, x)  # eight times an eighth, exact


def test_calls_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(12)
    tokens, top_k, hidden, n_experts = 300, 8, 520, 32
    ids = torch.from_numpy(ids_of(rng, tokens, top_k, n_experts)).cuda()
    x = rows_in(rng, tokens, hidden, torch.float16)
    w = torch.from_numpy(rng.random((tokens, top_k)).astype(np.float32)).cuda()

    def layer(stream=None):
        plan = experts.empty_plan(tokens, top_k, n_experts)
        rows = torch.empty((tokens * top_k, hidden), dtype=x.dtype, device="cuda")
        out = torch.empty_like(x)
        experts.sort(ids, n_experts, *plan, stream=stream)
        experts.gather(x, plan.inverse, plan.offsets, rows, stream)
        experts.combine(rows, w, plan.inverse, out, stream)
        return out, rows, plan

    want = layer()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = layer(side)
    side.synchronize()
    assert torch.equal(got[0], want[0])
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kept = layer()
    kept[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept[0], want[0])


def test_a_wrong_plan_stays_in_bounds():
    # places and offsets outside the buffers count as dropped or are clamped
    tokens, top_k, hidden = 40, 4, 256
    inverse = torch.full((tokens, top_k), 2 ** 30, dtype=torch.int32, device="cuda")
    inverse[:, 1] = -2 ** 31
    inverse[:, 2] = torch.arange(tokens, dtype=torch.int32, device="cuda")
    offsets = torch.full((9,), 2 ** 30, dtype=torch.int32, device="cuda")
    x = torch.randn((tokens, hidden), device="cuda")
    out, g = guarded_rows(tokens * top_k, hidden, hidden, 0, torch.float32)
    experts.gather(x, inverse, offsets, out)
    assert torch.equal(out[:tokens], x) and g.bands_intact()
    back = torch.empty_like(x)
    experts.combine(out, None, inverse, back)
    assert torch.equal(back, x)


def test_the_debug_build_declines_no_access(bq_lib):
    with _lib.use_library(build.build_debug_library()):
        codec.take_index_errors()
        for tokens, top_k, n_experts in SORTS[:9]:
            test_sort_is_the_stable_order_by_expert(tokens, top_k, n_experts, torch.int64)
        for shape in SHAPES:
            for name in TYPES:
                test_gather_copies_rows_to_their_places(name, shape)
                test_combine_sums_a_tokens_rows(name, shape, True)
                test_combine_sums_a_tokens_rows(name, shape, False)
                test_combine_grad_against_the_formula(name, shape)
        torch.cuda.synchronize()
        assert codec.take_index_errors() == 0


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("tokens,top_k,spare", [(17, 4, 0), (64, 8, 0), (64, 3, 5), (2000, 8, 0)])
def test_combine_grad_of_many_slots_without_columns(name, tokens, top_k, spare):
    # no columns: dweights are zeros, and nothing is read or written through the rows, whose
    # tensors have null pointers (or, with spare columns beside them, rows `spare` values apart)
    dtype = TYPES[name][0]
    ids = ids_of(np.random.default_rng(tokens), tokens, top_k, 5)
    offsets, order, inverse = device_plan(ids, 5)
    dout = torch.ones((tokens, spare), dtype=dtype, device="cuda")[:, :0]
    y = torch.ones((tokens * top_k, spare), dtype=dtype, device="cuda")[:, :0]
    around = torch.full((tokens * top_k, spare), 3.0, dtype=dtype, device="cuda")
    gw = Guarded(4 * tokens * top_k)
    dw = gw.view(torch.float32, (tokens, top_k))
    experts.combine_grad(dout, y, torch.full((tokens, top_k), float("nan"), device="cuda"), inverse, offsets,
                         around[:, :0], dw)
    assert not dw.any() and gw.bands_intact() and bool((around == 3.0).all())
