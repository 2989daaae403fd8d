"""The 4-bit products against the definition in 64 bits.

Tolerance. Products of an activation with a code are exact in binary32. A group's sum is
formed on the tensor cores in binary32 with at most one truncation per term, then scaled
and added: the error is at most (group + k / group + 16) * 2^-23 * sum |x w| to first order
(16: the column warps' sums and the scale's product), the factor 1.01 covering the rest.
One rounding to the output's type adds 2^-p * |result| (p = 8 for BF16, 11 for FP16) or
half its smallest subnormal.
"""
import numpy as np
import pytest
import torch

from block_quantized_wire_gb300 import _lib, build, codec, experts, w4
from tests.helpers import Guarded
from tests.test_gpu_experts import ids_of, plan_of

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (torch.bfloat16, 8, 2.0 ** -134), "f16": (torch.float16, 11, 2.0 ** -25)}


def make_weights(rng, lead, n, k, group, s_dtype, q_pad=0, s_pad=0):
    """Packed codes (all sixteen, -8 among them), scales, and the weights in 64 bits."""
    code = rng.integers(-8, 8, (*lead, n, k))
    packed = ((code[..., 0::2] & 15) | ((code[..., 1::2] & 15) << 4)).astype(np.uint8)
    wide = np.full((*lead, n, k // 2 + q_pad), 0x5A, np.uint8)
    wide[..., :k // 2] = packed
    s = torch.from_numpy((rng.standard_normal((*lead, n, k // group + s_pad)) * 0.02).astype(np.float32)).to(s_dtype)
    if s_pad:
        s[..., k // group:] = float("nan")
    s64 = s[..., :k // group].double().numpy()
    q = torch.from_numpy(wide).cuda()[..., :k // 2]
    return q, s.cuda()[..., :k // group], code * np.repeat(s64, group, axis=-1)


def make_x(rng, rows, k, dtype, pad=0):
    x = torch.from_numpy(rng.standard_normal((rows, k + pad)).astype(np.float32)).to(dtype)
    if pad:
        x[:, k:] = float("nan")
    x = x.cuda()[:, :k]
    return x, x.double().cpu().numpy()


def check(got, want, terms, k, group, p, tiny):
    bound = 1.01 * ((group + k // group + 16) * 2.0 ** -23 * terms + 2.0 ** -p * np.abs(want)) + tiny
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= bound), float((err - bound).max())


def guarded_out(rows, n, dtype, pad=0):
    g = Guarded(2 * rows * (n + pad))
    return g.view(dtype, (rows, n + pad))[:, :n], g


# rows, n, k, paddings of x, q, scales, out
DENSE = [(1, 1, 128, 0, 0, 0, 0), (1, 7168, 1024, 0, 0, 0, 0), (3, 96, 7168, 8, 0, 1, 0), (4, 47, 7168, 0, 16, 0, 5),
         (4, 200, 4096, 0, 0, 0, 0), (5, 33, 768, 0, 0, 0, 0), (16, 15400, 256, 0, 0, 0, 0),
         (1, 33, 7168, 0, 0, 0, 0), (2, 100, 384, 8, 16, 2, 3),
         (7, 65, 640, 0, 0, 0, 0), (8, 129, 2176, 16, 0, 1, 0), (9, 64, 1152, 0, 32, 3, 1), (16, 300, 896, 0, 0, 0, 0),
         (17, 31, 256, 0, 0, 0, 0), (32, 515, 4224, 0, 0, 0, 0), (33, 50, 1408, 0, 0, 0, 0), (100, 97, 512, 0, 0, 0, 0)]


@pytest.mark.parametrize("wide_scales", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("shape", DENSE)
def test_matvec(shape, name, group, wide_scales):
    rows, n, k, x_pad, q_pad, s_pad, out_pad = shape
    dtype, p, tiny = TYPES[name]
    rng = np.random.default_rng(rows * n + k + group)
    q, s, w = make_weights(rng, (), n, k, group, torch.float32 if wide_scales else dtype, q_pad, s_pad)
    x, x64 = make_x(rng, rows, k, dtype, x_pad)
    out, g = guarded_out(rows, n, dtype, out_pad)
    w4.matvec_w4(x, q, s, out)
    check(out, x64 @ w.T, np.abs(x64) @ np.abs(w).T, k, group, p, tiny)
    assert g.bands_intact()
    if out_pad:
        assert bool((g.view(torch.uint8).view(rows, -1)[:, 2 * n:] == Guarded.SENTINEL).all())


@pytest.mark.parametrize("k", [32, 64, 96, 160, 224, 1056])
def test_matvec_with_columns_that_end_inside_a_step(k):
    for group in (32, 64):
        if k % group:
            continue
        for s_dtype in (torch.bfloat16, torch.float32):
            rng = np.random.default_rng(k)
            q, s, w = make_weights(rng, (), 40, k, group, s_dtype)
            x, x64 = make_x(rng, 3, k, torch.bfloat16)
            out, g = guarded_out(3, 40, torch.bfloat16)
            w4.matvec_w4(x, q, s, out)
            check(out, x64 @ w.T, np.abs(x64) @ np.abs(w).T, k, group, 8, 2.0 ** -134)
            assert g.bands_intact()


# tokens, top_k, n_experts, n, k, group
EXPERTS = [(1, 1, 1, 16, 128, 128), (1, 8, 64, 100, 512, 32), (3, 2, 5, 33, 256, 64), (24, 6, 48, 70, 1024, 64),
           (32, 8, 8, 65, 384, 128), (50, 4, 3, 40, 640, 32), (200, 2, 300, 20, 256, 64), (700, 3, 9, 24, 128, 32),
           (2, 3, 1024, 16, 128, 64), (20, 1, 40, 50, 7168, 32), (3, 6, 20, 2000, 384, 128)]


@pytest.mark.parametrize("by_token", [True, False])
@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("shape", EXPERTS)
def test_matvec_experts(shape, name, by_token):
    tokens, top_k, n_experts, n, k, group = shape
    dtype, p, tiny = TYPES[name]
    rng = np.random.default_rng(tokens * 7 + n)
    ids = ids_of(rng, tokens, top_k, n_experts, skew=True)
    if top_k == 1:
        ids[::2] = 3  # one expert with far more rows than the average
    offsets, order, _ = plan_of(ids, n_experts)
    slots, kept = tokens * top_k, int(offsets[-1])
    q, s, w = make_weights(rng, (n_experts,), n, k, group, dtype if by_token else torch.float32)
    x, x64 = make_x(rng, tokens if by_token else slots, k, dtype)
    if not by_token:
        x[kept:] = float("nan")  # rows at places that no slot takes are not read
    out, g = guarded_out(slots, n, dtype)
    w4.matvec_w4_experts(x, q, s, torch.from_numpy(offsets).cuda(), out,
                         order=torch.from_numpy(order).cuda() if by_token else None, top_k=top_k)
    want, terms = np.zeros((slots, n)), np.zeros((slots, n))
    for e in range(n_experts):
        at = np.arange(offsets[e], offsets[e + 1])
        rows = x64[order[at] // top_k if by_token else at]
        want[at], terms[at] = rows @ w[e].T, np.abs(rows) @ np.abs(w[e]).T
    check(out, want, terms, k, group, p, tiny)
    assert not out[kept:].any() and g.bands_intact()


@pytest.mark.parametrize("rows", [4, 5, 12])
@pytest.mark.parametrize("name", list(TYPES))
def test_an_infinite_row_leaves_the_others_alone(rows, name):
    rng = np.random.default_rng(3)
    dtype = TYPES[name][0]
    q, s, w = make_weights(rng, (), 48, 256, 32, dtype)
    x, _ = make_x(rng, rows, 256, dtype)
    clean = torch.empty((rows, 48), dtype=dtype, device="cuda")
    w4.matvec_w4(x, q, s, clean)
    x[2, 7], x[3, 9] = float("inf"), float("nan")
    out = torch.empty_like(clean)
    w4.matvec_w4(x, q, s, out)
    code = torch.from_numpy(w[:, 7]).cuda()
    assert torch.equal(out[2] == float("inf"), code > 0) and torch.equal(out[2] == float("-inf"), code < 0)
    assert torch.equal(out[2].isnan(), code == 0) and bool(out[3].isnan().all())
    for r in set(range(rows)) - {2, 3}:
        assert torch.equal(out[r], clean[r])


def test_values_far_below_their_rows_largest():
    # through FP16 a BF16 row's values below 2^-31 of its largest are off by at most 2^-39 of it
    rng = np.random.default_rng(21)
    k, n = 1024, 64
    q, s, w = make_weights(rng, (), n, k, 64, torch.bfloat16)
    x32 = (rng.standard_normal((3, k)) * 2.0 ** rng.integers(-45, 0, (3, k))).astype(np.float32)
    x32[:, 100] = [2.0 ** 20, 3.0e38, 2.0 ** -100]
    x = torch.from_numpy(x32).to(torch.bfloat16).cuda()
    x64 = x.double().cpu().numpy()
    for cleared in (False, True):
        if cleared:
            q[:, 50] = q[:, 50] & 0xF0  # column 100's codes: the largest value takes no part
            w[:, 100] = 0.0
        out = torch.empty((3, n), dtype=torch.bfloat16, device="cuda")
        w4.matvec_w4(x, q, s, out)
        terms = np.abs(x64) @ np.abs(w).T
        terms += 2.0 ** -16 / (64 + 16 + 16) * np.abs(x64).max(1)[:, None] * np.abs(w).sum(1)  # 2^-39 in check's unit
        check(out, x64 @ w.T, terms, k, 64, 8, 2.0 ** -134)


def staged_case(name, s_dtype, lead, n, k, group, seed):
    """Weights large enough for the kernel that keeps rows of x in shared memory, drawn on the
    GPU, and a function that gives an expert's weights in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    code = torch.randint(-8, 8, (*lead, n, k), generator=g, device="cuda", dtype=torch.int8)
    q = ((code[..., 0::2] & 15) | ((code[..., 1::2] & 15) << 4)).view(torch.uint8)
    s = (torch.randn((*lead, n, k // group), generator=g, device="cuda") * 0.02).to(s_dtype)

    def weights(*at):
        return code[at].double() * s[at].double().repeat_interleave(group, dim=-1)
    return g, q, s, weights


@pytest.mark.parametrize("wide_range", [False, True])
@pytest.mark.parametrize("name,wide_scales,k,group", [("bf16", False, 4096, 32), ("bf16", True, 4160, 64),
                                                      ("f16", False, 4352, 128), ("f16", True, 7200, 32)])
def test_one_row_times_many(name, wide_scales, k, group, wide_range):
    dtype, p, tiny = TYPES[name]
    n = 19500
    g, q, s, weights = staged_case(name, torch.float32 if wide_scales else dtype, (), n, k, group, k)
    x = torch.randn((1, k), generator=g, device="cuda")
    if wide_range and name == "bf16":
        x *= 2.0 ** torch.randint(-45, 0, (1, k), generator=g, device="cuda")
        x[0, 100] = 2.0 ** 30
    x = x.to(dtype)
    out, guard = guarded_out(1, n, dtype)
    w4.matvec_w4(x, q, s, out)
    w, x64 = weights(), x.double()
    want, terms = x64 @ w.T, x64.abs() @ w.abs().T
    if name == "bf16":  # through FP16: 2^-39 of the largest for each value, in check's unit
        terms += 2.0 ** -16 / (group + k // group + 16) * x64.abs().max() * w.abs().sum(1)
    check(out, want.cpu().numpy(), terms.cpu().numpy(), k, group, p, tiny)
    assert guard.bands_intact()


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("k", [4096, 7168])
def test_experts_with_one_row_on_average(name, k):
    # 12 tokens over 24 experts of 1650 rows: the kernel expects one row an expert, and one
    # expert has nine, more than its shared memory holds at once
    dtype, p, tiny = TYPES[name]
    group, n, n_experts = 64, 1650, 24
    g, q, s, weights = staged_case(name, dtype, (n_experts,), n, k, group, 3)
    ids = np.array([[3]] * 5 + [[0]] + [[3]] * 4 + [[23], [40]])
    offsets, order, _ = plan_of(ids, n_experts)
    x = torch.randn((12, k), generator=g, device="cuda").to(dtype)
    out, guard = guarded_out(12, n, dtype)
    w4.matvec_w4_experts(x, q, s, torch.from_numpy(offsets).cuda(), out, order=torch.from_numpy(order).cuda(), top_k=1)
    want, terms = torch.zeros((12, n), dtype=torch.float64), torch.zeros((12, n), dtype=torch.float64)
    for e in (0, 3, 23):
        at = slice(int(offsets[e]), int(offsets[e + 1]))
        rows, w = x[torch.from_numpy(order[at]).cuda().long()].double(), weights(e)
        want[at], terms[at] = (rows @ w.T).cpu(), (rows.abs() @ w.abs().T).cpu()
        if name == "bf16":
            few = 2.0 ** -16 / (group + k // group + 16) * rows.abs().max() * w.abs().sum(1)
            terms[at] += few.cpu()
    check(out, want.numpy(), terms.numpy(), k, group, p, tiny)
    assert not out[11].any() and guard.bands_intact()


@pytest.mark.parametrize("rows", [1, 4, 6])
@pytest.mark.parametrize("name,wide_scales,k,group", [("bf16", False, 4160, 64), ("bf16", True, 4192, 32),
                                                      ("f16", False, 4224, 128), ("f16", True, 4160, 64)])
def test_many_items_of_several_steps(name, wide_scales, k, group, rows):
    # so many weight rows that a warp takes two row tiles, and several steps of each item; an odd
    # number of scales a row, and columns that end inside a step
    dtype, p, tiny = TYPES[name]
    n = 7210
    g, q, s, weights = staged_case(name, torch.float32 if wide_scales else dtype, (), n, k, group, k + rows)
    x = torch.randn((rows, k), generator=g, device="cuda").to(dtype)
    out, guard = guarded_out(rows, n, dtype)
    w4.matvec_w4(x, q, s, out)
    w, x64 = weights(), x.double()
    check(out, (x64 @ w.T).cpu().numpy(), (x64.abs() @ w.abs().T).cpu().numpy(), k, group, p, tiny)
    assert guard.bands_intact()


@pytest.mark.parametrize("name", list(TYPES))
def test_experts_with_many_items_of_several_steps(name):
    dtype, p, tiny = TYPES[name]
    group, n, k, n_experts = 64, 2410, 4160, 8
    g, q, s, weights = staged_case(name, dtype, (n_experts,), n, k, group, 5)
    rng = np.random.default_rng(5)
    ids = ids_of(rng, 16, 2, n_experts, skew=True)
    offsets, order, _ = plan_of(ids, n_experts)
    x = torch.randn((16, k), generator=g, device="cuda").to(dtype)
    out, guard = guarded_out(32, n, dtype)
    w4.matvec_w4_experts(x, q, s, torch.from_numpy(offsets).cuda(), out, order=torch.from_numpy(order).cuda(), top_k=2)
    want, terms = torch.zeros((32, n), dtype=torch.float64), torch.zeros((32, n), dtype=torch.float64)
    for e in range(n_experts):
        at = slice(int(offsets[e]), int(offsets[e + 1]))
        if at.start < at.stop:
            rows, w = x[torch.from_numpy(order[at] // 2).cuda().long()].double(), weights(e)
            want[at], terms[at] = (rows @ w.T).cpu(), (rows.abs() @ w.abs().T).cpu()
    check(out, want.numpy(), terms.numpy(), k, group, p, tiny)
    assert not out[int(offsets[-1]):].any() and guard.bands_intact()


@pytest.mark.parametrize("name", list(TYPES))
def test_a_row_of_infinities_times_many(name):
    dtype = TYPES[name][0]
    g, q, s, weights = staged_case(name, dtype, (), 19500, 4096, 32, 8)
    x = torch.randn((1, 4096), generator=g, device="cuda").to(dtype)
    x[0, 7] = float("inf")
    out = torch.empty((1, 19500), dtype=dtype, device="cuda")
    w4.matvec_w4(x, q, s, out)
    w = weights()[:, 7]
    assert torch.equal(out[0] == float("inf"), w > 0) and torch.equal(out[0] == float("-inf"), w < 0)
    x[0, 7] = float("nan")
    w4.matvec_w4(x, q, s, out)
    assert bool(out.isnan().all())


def test_rows_do_not_depend_on_their_company():
    # row 0 alone, with 7 and with 31 others, and repeated calls: the same bits wherever the
    # same kernel runs, and within one launch wherever the row stands
    rng = np.random.default_rng(4)
    q, s, _ = make_weights(rng, (), 200, 2048, 64, torch.float16)
    x, _ = make_x(rng, 8, 2048, torch.float16)
    x[5] = x[0]
    outs = []
    for _ in range(3):
        out = torch.empty((8, 200), dtype=torch.float16, device="cuda")
        w4.matvec_w4(x, q, s, out)
        outs.append(out)
    one = torch.empty((1, 200), dtype=torch.float16, device="cuda")
    w4.matvec_w4(x[:1], q, s, one)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert torch.equal(outs[0][0], outs[0][5]) and torch.equal(one[0], outs[0][0])


def test_calls_with_more_and_less_shared_memory_in_turn():
    # the kernel's shared memory grows with the number of experts: a call with few experts must
    # not take the limit away from the one with many
    rng = np.random.default_rng(31)
    for n_experts in (900, 3, 900, 40, 900, 3):
        q = torch.full((n_experts, 32, 64), 0x11, dtype=torch.uint8, device="cuda")
        s = torch.ones((n_experts, 32, 2), dtype=torch.bfloat16, device="cuda")
        x = torch.from_numpy(rng.integers(0, 2, (1, 128)).astype(np.float32)).to(torch.bfloat16).cuda()
        offsets = torch.ones(n_experts + 1, dtype=torch.int32, device="cuda")
        offsets[0] = 0
        out = torch.empty((1, 32), dtype=torch.bfloat16, device="cuda")
        w4.matvec_w4_experts(x, q, s, offsets, out)
        assert bool((out == x.sum()).all())


def test_no_rows_no_columns_and_an_empty_sum():
    e = torch.empty
    q, s = e((8, 64), dtype=torch.uint8, device="cuda"), torch.ones((8, 1), dtype=torch.bfloat16, device="cuda")
    w4.matvec_w4(e((0, 128), dtype=torch.bfloat16, device="cuda"), q, s, e((0, 8), dtype=torch.bfloat16, device="cuda"))
    w4.matvec_w4(e((3, 128), dtype=torch.bfloat16, device="cuda"), q[:0], s[:0],
                 e((3, 0), dtype=torch.bfloat16, device="cuda"))
    out = torch.full((3, 8), 7.0, dtype=torch.bfloat16, device="cuda")
    w4.matvec_w4(e((3, 0), dtype=torch.bfloat16, device="cuda"), e((8, 0), dtype=torch.uint8, device="cuda"),
                 e((8, 0), dtype=torch.bfloat16, device="cuda"), out)
    assert not out.any()


def test_weights_past_2_32_bytes():
    # 300 experts of 16 MB: the last one's codes start past 2^32 bytes
    n_experts, n, k, group = 300, 4096, 8192, 128
    q = torch.zeros((n_experts, n, k // 2), dtype=torch.uint8, device="cuda")
    s = torch.ones((n_experts, n, k // group), dtype=torch.bfloat16, device="cuda")
    q[-1] = 0x21  # codes 1 (even columns) and 2 (odd columns)
    ids = np.array([[299, 0]])
    offsets, order, _ = plan_of(ids, n_experts)
    x = torch.ones((1, k), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((2, n), dtype=torch.bfloat16, device="cuda")
    w4.matvec_w4_experts(x, q, s, torch.from_numpy(offsets).cuda(), out, order=torch.from_numpy(order).cuda(), top_k=2)
    assert not out[0].any() and bool((out[1] == 3 * k // 2).all())


def test_a_wrong_plan_stays_in_bounds():
    rng = np.random.default_rng(9)
    q, s, _ = make_weights(rng, (4,), 40, 256, 64, torch.bfloat16)
    x, _ = make_x(rng, 6, 256, torch.bfloat16)
    out, g = guarded_out(12, 40, torch.bfloat16)
    for offsets, order in (([0, 2 ** 30, 3, 2 ** 30, 2 ** 31 - 1], [2 ** 30] * 12), ([-5, 4, -9, 12, -1], [-1] * 12)):
        w4.matvec_w4_experts(x, q, s, torch.tensor(offsets, dtype=torch.int32, device="cuda"), out,
                             order=torch.tensor(order, dtype=torch.int32, device="cuda"), top_k=2)
        torch.cuda.synchronize()
        assert g.bands_intact()


def test_the_debug_build_declines_no_access(bq_lib):
    with _lib.use_library(build.build_debug_library()):
        codec.take_index_errors()
        for shape in DENSE:
            for group in (32, 128):
                test_matvec(shape, "bf16", group, False)
                test_matvec(shape, "f16", group, True)
        for shape in EXPERTS:
            test_matvec_experts(shape, "bf16", True)
            test_matvec_experts(shape, "f16", False)
        test_one_row_times_many("bf16", True, 4160, 64, False)
        test_experts_with_one_row_on_average("f16", 7168)
        test_many_items_of_several_steps("bf16", False, 4160, 64, 6)
        test_many_items_of_several_steps("f16", True, 4160, 64, 4)
        test_experts_with_many_items_of_several_steps("bf16")
        torch.cuda.synchronize()
        assert codec.take_index_errors() == 0


# Rows kept in shared memory (one row on average, many long weight rows). Their values and
# sums have the range and precision of rows read directly: products are exact, so check's own
# bound holds without an allowance.
STAGED = [("bf16", False, 4096, 32), ("bf16", True, 4160, 64), ("bf16", False, 7168, 128), ("f16", True, 4096, 32)]


@pytest.mark.parametrize("name,wide_scales,k,group", STAGED)
def test_one_row_whose_largest_value_takes_no_part(name, wide_scales, k, group):
    dtype, p, tiny = TYPES[name]
    n = 19500
    g, q, s, weights = staged_case(name, torch.float32 if wide_scales else dtype, (), n, k, group, k + 1)
    q[:, 50] &= 0xF0  # column 100's codes
    w = weights()
    w[:, 100] = 0.0
    x = torch.randn((1, k), generator=g, device="cuda") * 2.0 ** torch.randint(-12, 0, (1, k), generator=g, device="cuda")
    x[0, 100] = 2.0 ** 14
    x = x.to(dtype)
    if name == "bf16":
        x *= 2.0 ** -40
        x[0, 100] = 2.0 ** 30
    out, guard = guarded_out(1, n, dtype)
    w4.matvec_w4(x, q, s, out)
    x64 = x.double()
    check(out, (x64 @ w.T).cpu().numpy(), (x64.abs() @ w.abs().T).cpu().numpy(), k, group, p, tiny)
    assert guard.bands_intact()


@pytest.mark.parametrize("group", [32, 128])
def test_an_experts_row_whose_largest_value_takes_no_part(group):
    dtype, p, tiny = TYPES["bf16"]
    n, k, n_experts = 3000, 4096, 24
    g, q, s, weights = staged_case("bf16", dtype, (n_experts,), n, k, group, 13)
    s[..., 100 // group] = 0.0  # the scales of the largest value's group
    ids = np.array([[3], [0], [3], [23], [3], [3], [3]])
    offsets, order, _ = plan_of(ids, n_experts)
    x = torch.randn((7, k), generator=g, device="cuda").to(dtype) * 2.0 ** -45
    x[:, 100] = 3.0e38
    out, guard = guarded_out(7, n, dtype)
    w4.matvec_w4_experts(x, q, s, torch.from_numpy(offsets).cuda(), out, order=torch.from_numpy(order).cuda(), top_k=1)
    want, terms = torch.zeros((7, n), dtype=torch.float64), torch.zeros((7, n), dtype=torch.float64)
    for e in (0, 3, 23):
        at = slice(int(offsets[e]), int(offsets[e + 1]))
        rows, w = x[torch.from_numpy(order[at]).cuda().long()].double(), weights(e)
        want[at], terms[at] = (rows @ w.T).cpu(), (rows.abs() @ w.abs().T).cpu()
    check(out, want.numpy(), terms.numpy(), k, group, p, tiny)
    assert guard.bands_intact()


@pytest.mark.parametrize("wide_scales", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_a_staged_rows_sums_do_not_overflow_before_the_result(group, wide_scales):
    # 4096 ones times codes of 7 and scales of 2^112: 7 * 2^124, exact in BF16
    k, n = 4096, 19500
    q = torch.full((n, k // 2), 0x77, dtype=torch.uint8, device="cuda")
    s = torch.full((n, k // group), 2.0 ** 112, dtype=torch.float32 if wide_scales else torch.bfloat16, device="cuda")
    x = torch.ones((1, k), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((1, n), dtype=torch.bfloat16, device="cuda")
    w4.matvec_w4(x, q, s, out)
    assert bool((out.double() == 7 * 2.0 ** 124).all())
    few = torch.empty((1, 64), dtype=torch.bfloat16, device="cuda")
    w4.matvec_w4(x, q[:64], s[:64], few)
    assert torch.equal(few, out[:, :64])
    q, s = (t[:n // 3].expand(6, -1, -1).contiguous() for t in (q, s))
    rows = torch.empty((3, n // 3), dtype=torch.bfloat16, device="cuda")  # a row for each of the first three experts
    offsets = torch.tensor([0, 1, 2, 3, 3, 3, 3], dtype=torch.int32, device="cuda")
    w4.matvec_w4_experts(x.expand(3, k).contiguous(), q, s, offsets, rows)
    assert bool((rows == out[0, 0]).all())


# 912 items of 16 weight rows, three rounds of the CTAs, where two-tile items would take two
# longer ones: staged rows of lengths that end inside a step, with odd numbers of scales
ODD_STAGED = [("bf16", False, 4160, 64), ("bf16", True, 7200, 32), ("bf16", False, 7200, 32), ("f16", False, 4160, 64)]


@pytest.mark.parametrize("name,wide_scales,k,group", ODD_STAGED)
def test_one_row_of_odd_length_times_many(name, wide_scales, k, group):
    dtype, p, tiny = TYPES[name]
    n = 14587
    g, q, s, weights = staged_case(name, torch.float32 if wide_scales else dtype, (), n, k, group, k + 2)
    x = torch.randn((1, k), generator=g, device="cuda").to(dtype)
    out, guard = guarded_out(1, n, dtype)
    w4.matvec_w4(x, q, s, out)
    w, x64 = weights(), x.double()
    check(out, (x64 @ w.T).cpu().numpy(), (x64.abs() @ w.abs().T).cpu().numpy(), k, group, p, tiny)
    assert guard.bands_intact()


@pytest.mark.parametrize("name,wide_scales,k,group", ODD_STAGED)
def test_experts_rows_of_odd_length_beyond_the_staged_ones(name, wide_scales, k, group):
    # 24 slots over 48 experts, one of which has ten rows, more than are staged at once
    dtype, p, tiny = TYPES[name]
    n, n_experts = 599, 48
    g, q, s, weights = staged_case(name, torch.float32 if wide_scales else dtype, (n_experts,), n, k, group, k + 3)
    ids = np.array([[7]] * 5 + [[e] for e in (0, 47, 60, 9, 33, 2, 2, 18, 5)] + [[7]] * 5 + [[e] for e in range(20, 25)])
    offsets, order, _ = plan_of(ids, n_experts)
    x = torch.randn((24, k), generator=g, device="cuda").to(dtype)
    out, guard = guarded_out(24, n, dtype)
    w4.matvec_w4_experts(x, q, s, torch.from_numpy(offsets).cuda(), out, order=torch.from_numpy(order).cuda(), top_k=1)
    want, terms = torch.zeros((24, n), dtype=torch.float64), torch.zeros((24, n), dtype=torch.float64)
    for e in range(n_experts):
        at = slice(int(offsets[e]), int(offsets[e + 1]))
        if at.start < at.stop:
            rows, w = x[torch.from_numpy(order[at]).cuda().long()].double(), weights(e)
            want[at], terms[at] = (rows @ w.T).cpu(), (rows.abs() @ w.abs().T).cpu()
    check(out, want.numpy(), terms.numpy(), k, group, p, tiny)
    assert not out[int(offsets[-1]):].any() and guard.bands_intact()


def test_staged_rows_in_the_debug_build_decline_no_access(bq_lib):
    with _lib.use_library(build.build_debug_library()):
        codec.take_index_errors()
        for case in ODD_STAGED:
            test_one_row_of_odd_length_times_many(*case)
            test_experts_rows_of_odd_length_beyond_the_staged_ones(*case)
        for case in STAGED:
            test_one_row_whose_largest_value_takes_no_part(*case)
        torch.cuda.synchronize()
        assert codec.take_index_errors() == 0


@pytest.mark.parametrize("n,rows", [(48, 1), (48, 6), (48, 12), (19500, 1)])
@pytest.mark.parametrize("name", list(TYPES))
def test_rows_of_subnormal_values(name, n, rows):
    # the smallest values that x can hold, with FP32 scales that bring the result up: products
    # and sums are exact multiples of x's smallest, so check's bound holds as it stands
    dtype, p, tiny = TYPES[name]
    k, group = 4096, 64
    g, q, s, weights = staged_case(name, torch.float32, (), n, k, group, n + rows)
    smallest = 2.0 ** -133 if name == "bf16" else 2.0 ** -24
    s.copy_(s.abs().add_(0.01) * (2.0 ** 60 if name == "bf16" else 1.0))
    x64 = torch.randint(-7, 8, (rows, k), generator=g, device="cuda").double() * smallest
    x = x64.to(dtype)
    assert torch.equal(x.double(), x64)
    out, guard = guarded_out(rows, n, dtype)
    w4.matvec_w4(x, q, s, out)
    w = weights()
    check(out, (x64 @ w.T).cpu().numpy(), (x64.abs() @ w.abs().T).cpu().numpy(), k, group, p, tiny)
    assert guard.bands_intact()


def test_equal_rows_give_equal_results_in_every_form():
    # a row repeated at other places of one launch, and the launch repeated: the same bits
    for rows, n, k in ((32, 200, 2048), (32, 40000, 1024), (4, 30000, 2048), (8, 4864, 4096)):
        g, q, s, _ = staged_case("bf16", torch.bfloat16, (), n, k, 32, rows)
        x = torch.randn((rows, k), generator=g, device="cuda").to(torch.bfloat16)
        x[rows - 1], x[rows // 2] = x[0], x[0]
        outs = [torch.empty((rows, n), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        for out in outs:
            w4.matvec_w4(x, q, s, out)
        assert torch.equal(outs[0], outs[1])
        assert torch.equal(outs[0][0], outs[0][rows - 1]) and torch.equal(outs[0][0], outs[0][rows // 2])
