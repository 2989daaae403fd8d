"""The expert layer's calls together: a decode step over simulated ranks and the training
form with its gradients, and the 4-bit quantization of expert weights bit for bit."""
import numpy as np
import pytest
import torch

from block_quantized_wire_gb300 import _lib, build, codec, moe, topology, w4
from tests.helpers import Guarded

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def quantized(x, group, s_dtype):
    """The definition with numpy's binary32 arithmetic: packed codes, scales, codes."""
    v = x.float().cpu().numpy().reshape(*x.shape[:-1], -1, group)
    amax = np.abs(v).max(-1)
    s = torch.from_numpy((amax / np.float32(7)).astype(np.float32)).to(s_dtype)
    s32 = s.float().numpy()
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        code = np.clip(np.rint(v / s32[..., None]), -7, 7)
    code = np.where(s32[..., None] > 0, code, 0).astype(np.int64).reshape(x.shape)
    return ((code[..., 0::2] & 15) | ((code[..., 1::2] & 15) << 4)).astype(np.uint8), s, code


@pytest.mark.parametrize("s_name", list(TYPES))
@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quant_w4_is_bit_exact(name, s_name, group):
    rng = np.random.default_rng(group)
    for lead, n, k in (((), 1, 128), ((), 37, 1152), ((3,), 20, 384)):
        x32 = rng.standard_normal((*lead, n, k)) * 10.0 ** rng.uniform(-3, 3, (*lead, n, 1))
        x32[..., 0, :group] = 0.0
        x32[..., -1, :group] = 2.0 ** -24  # scales that underflow in FP16
        x = torch.from_numpy(x32.astype(np.float32)).to(TYPES[name]).cuda()
        gq, gs = Guarded(x.numel() // 2), Guarded(x.numel() // group * (4 if s_name == "f32" else 2))
        q = gq.view(torch.uint8, (*lead, n, k // 2))
        s = gs.view(TYPES[s_name], (*lead, n, k // group))
        w4.quant_w4(x, q, s)
        want_q, want_s, _ = quantized(x, group, TYPES[s_name])
        assert np.array_equal(q.cpu().numpy(), want_q)
        assert torch.equal(s.cpu(), want_s)
        assert gq.bands_intact() and gs.bands_intact()


def test_quant_w4_in_the_debug_build_declines_no_access(bq_lib):
    with _lib.use_library(build.build_debug_library()):
        codec.take_index_errors()
        for name in TYPES:
            test_quant_w4_is_bit_exact(name, "f32", 64)
        torch.cuda.synchronize()
        assert codec.take_index_errors() == 0


def dequantized(pair):
    q, s = (t.cpu() for t in pair)
    q = q.to(torch.int64)
    code = torch.stack([q & 15, q >> 4], dim=-1).flatten(-2)
    code = torch.where(code > 7, code - 16, code)
    return code.double() * s.double().repeat_interleave(code.shape[-1] // s.shape[-1], dim=-1)


@pytest.mark.parametrize("mode", ["", "i8_a2a", "mx_a2a", "i8_ring"])
def test_decode_layer_over_four_ranks(mode):
    torch.manual_seed(3)
    tokens, top_k, n_ranks, each, hidden, inner = 8, 4, 4, 6, 256, 128
    n_experts = n_ranks * each
    x = torch.randn(tokens, hidden, device="cuda").to(torch.bfloat16)
    top, ids = torch.randn(tokens, n_experts, device="cuda").topk(top_k, dim=1)
    weights = torch.softmax(top, dim=1)
    gate_up = (torch.randn(n_experts, 2 * inner, hidden, device="cuda") * hidden ** -0.5).to(torch.bfloat16)
    down = (torch.randn(n_experts, hidden, inner, device="cuda") * inner ** -0.5).to(torch.bfloat16)
    ranks = [moe.quantize_experts(r * each, gate_up[r * each:(r + 1) * each].contiguous(),
                                  down[r * each:(r + 1) * each].contiguous()) for r in range(n_ranks)]
    out = moe.decode_layer(x, ids, weights, ranks, mode)
    got = torch.cat(out).double().cpu()
    gu, dn = (torch.cat([dequantized(getattr(w, f)) for w in ranks]) for f in ("gate_up", "down"))
    want = torch.zeros(tokens, hidden, dtype=torch.float64)
    x64, w64 = x.double().cpu(), weights.double().cpu()
    for t in range(tokens):
        for j in range(top_k):
            e = int(ids[t, j])
            a = gu[e] @ x64[t]
            g, u = a[:inner], a[inner:]
            want[t] += w64[t, j] * (dn[e] @ (g * torch.sigmoid(g) * u))
    # BF16 roundings of the products, the activation, the parts (2^-8 each, five deep) and, per
    # wire hop, a payload step of amax / 127 / 2 (INT8) or 2^-4 of the value (E4M3)
    amax = float(want.abs().max())
    wire = {"": 0.0, "i8_a2a": 5 / 254, "i8_ring": 4 / 254, "mx_a2a": 2 / 16}[mode]
    assert float((got - want).abs().max()) <= (5 * 2.0 ** -8 * 4 + wire * 2) * amax


def test_training_form_and_its_gradients():
    # a linear map per expert, so that the plain layer can be differentiated in 64 bits
    torch.manual_seed(4)
    tokens, top_k, n_experts, first, hidden = 50, 3, 5, 4, 96
    x = torch.randn(tokens, hidden, device="cuda")
    ids = torch.randint(0, 16, (tokens, top_k), device="cuda")
    weights = torch.rand(tokens, top_k, device="cuda")
    maps = torch.randn(n_experts, hidden, hidden, device="cuda") * hidden ** -0.5
    dout = torch.randn(tokens, hidden, device="cuda")

    def by_expert(rows, offsets, m):
        ends = offsets.tolist()
        out = torch.zeros_like(rows)
        for e in range(n_experts):
            out[ends[e]:ends[e + 1]] = (rows[ends[e]:ends[e + 1]].double() @ m[e].double()).float()
        return out

    p = moe.part(x, ids, weights, first, n_experts, lambda rows, offsets: by_expert(rows, offsets, maps))
    dx, dw = moe.part_grad(dout, weights, p, lambda d, rows, offsets: by_expert(d, offsets, maps.transpose(1, 2)))
    x64, w64 = (t.double().cpu().requires_grad_() for t in (x, weights))
    m64, id_cpu = maps.double().cpu(), ids.cpu() - first
    here = (id_cpu >= 0) & (id_cpu < n_experts)
    each = torch.einsum("th,tjhk->tjk", x64, m64[id_cpu.clamp(0, n_experts - 1)])
    want = (each * (w64 * here)[..., None]).sum(1)
    want.backward(dout.double().cpu())
    # binary32 sums of at most hidden + top_k + 2 terms, each term below the largest product
    for got, ref, n in ((p.out, want.detach(), top_k + 2), (dx, x64.grad, top_k + 3), (dw, w64.grad, hidden + 3)):
        bound = 2.0 ** -23 * n * float(ref.abs().max()) * 8 + 1e-12
        assert float((got.double().cpu() - ref).abs().max()) <= bound
    assert not dw.cpu()[~here].any()


@pytest.mark.parametrize("mode", ["i8_ring", "i8_a2a", "i8_ag", "mx_ring", "mx_a2a", "e4m3_ag"])
def test_decode_layer_returns_what_the_modes_owners_hold(mode):
    torch.manual_seed(5)
    tokens, n_ranks, hidden, inner = 8, 4, 256, 64
    x = torch.randn(tokens, hidden, device="cuda").to(torch.bfloat16)
    top, ids = torch.randn(tokens, 2 * n_ranks, device="cuda").topk(3, dim=1)
    weights = torch.softmax(top, dim=1)
    ranks = [moe.quantize_experts(2 * r, *((torch.randn(2, *shape, device="cuda") / 16).to(torch.bfloat16)
                                           for shape in ((2 * inner, hidden), (hidden, inner)))) for r in range(n_ranks)]
    parts = [moe.decode_part(x, ids, weights, w) for w in ranks]
    owned = topology.MODES[mode](parts)[2]
    want = owned if isinstance(owned, torch.Tensor) else torch.cat(owned)
    assert torch.equal(torch.cat(moe.decode_layer(x, ids, weights, ranks, mode)), want)
