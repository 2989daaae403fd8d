"""The expert-layer calls without a GPU: the C ABI's refusals (before any CUDA call; the
fake pointers are never dereferenced) and the binding's checks of tensors."""
import os
import subprocess
import sys

import pytest
import torch

from block_quantized_wire_gb300 import build, experts, w4

OK, NULL, SHAPE, ALIGN, ALIAS = range(5)
A = 0x7F0000000000  # a 256-byte-aligned fake device address
M = 0x1000000
BF16, F16, F32 = range(3)


def test_sort_rejections(bq_lib):
    def f(ids=A, wide=0, tokens=100, top_k=8, n=64, offsets=A + M, order=A + 2 * M, inverse=A + 3 * M, ws=A + 4 * M):
        return bq_lib.bq_expert_sort(ids, wide, tokens, top_k, n, offsets, order, inverse, ws, None)
    assert f(tokens=-1) == SHAPE
    assert f(top_k=0) == SHAPE and f(top_k=65) == SHAPE
    assert f(n=0) == SHAPE and f(n=1025) == SHAPE
    assert f(tokens=2 ** 28) == SHAPE  # 2^31 slots
    for name in ("ids", "offsets", "order", "inverse", "ws"):
        assert f(**{name: None}) == NULL
    assert f(ids=A + 2) == ALIGN and f(ids=A + 4, wide=1) == ALIGN
    for name, base in (("offsets", 1), ("order", 2), ("inverse", 3), ("ws", 4)):
        assert f(**{name: A + base * M + 2}) == ALIGN
    assert f(order=A + 16) == ALIAS and f(inverse=A + 2 * M + 3196) == ALIAS
    assert f(ws=A + M + 256) == ALIAS and f(ws=A + 3 * M - 4) == ALIAS


def test_gather_rejections(bq_lib):
    def f(x=A, type=BF16, tokens=10, hidden=64, ld_x=64, inverse=A + M, top_k=4, offsets=A + 2 * M, n=8, out=A + 3 * M,
          ld_out=64):
        return bq_lib.bq_expert_gather(x, type, tokens, hidden, ld_x, inverse, top_k, offsets, n, out, ld_out, None)
    assert f(tokens=0, x=None) == OK and f(hidden=0, out=None) == OK  # nothing to do, no launch
    assert f(type=3) == SHAPE and f(type=-1) == SHAPE and f(tokens=-1) == SHAPE and f(hidden=-1) == SHAPE
    assert f(top_k=0) == SHAPE and f(n=0) == SHAPE and f(ld_x=63) == SHAPE and f(ld_out=63) == SHAPE
    for name in ("x", "inverse", "offsets", "out"):
        assert f(**{name: None}) == NULL
    assert f(x=A + 1) == ALIGN and f(x=A + 2, type=F32) == ALIGN and f(out=A + 3 * M + 1) == ALIGN
    assert f(inverse=A + M + 2) == ALIGN and f(offsets=A + 2 * M + 2) == ALIGN
    assert f(out=A + 1278) == ALIAS and f(out=A + M + 156) == ALIAS and f(out=A + 2 * M) == ALIAS


def test_combine_rejections(bq_lib):
    def f(y=A, type=F16, ld_y=64, weights=A + M, inverse=A + 2 * M, tokens=10, top_k=4, hidden=64, out=A + 3 * M,
          ld_out=64):
        return bq_lib.bq_expert_combine(y, type, ld_y, weights, inverse, tokens, top_k, hidden, out, ld_out, None)
    assert f(tokens=0, y=None) == OK and f(hidden=0, y=None) == OK
    assert f(type=9) == SHAPE and f(tokens=-1) == SHAPE and f(top_k=65) == SHAPE and f(ld_y=63) == SHAPE
    assert f(ld_out=1) == SHAPE
    for name in ("y", "inverse", "out"):
        assert f(**{name: None}) == NULL
    assert f(y=A + 1) == ALIGN and f(weights=A + M + 2) == ALIGN and f(inverse=A + 2 * M + 1) == ALIGN
    assert f(out=A) == ALIAS and f(out=A + M + 158) == ALIAS and f(out=A + 2 * M - 2) == ALIAS


def test_combine_grad_rejections(bq_lib):
    def f(dout=A, type=BF16, ld_d=64, y=A + M, ld_y=64, weights=A + 2 * M, inverse=A + 3 * M, offsets=A + 4 * M, n=8,
          tokens=10, top_k=4, hidden=64, dy=A + 5 * M, ld_dy=64, dw=A + 6 * M):
        return bq_lib.bq_expert_combine_grad(dout, type, ld_d, y, ld_y, weights, inverse, offsets, n, tokens, top_k,
                                             hidden, dy, ld_dy, dw, None)
    assert f(tokens=0, dout=None) == OK
    assert f(type=4) == SHAPE and f(n=1025) == SHAPE and f(ld_dy=63) == SHAPE and f(ld_d=2) == SHAPE
    for name in ("dout", "y", "weights", "inverse", "offsets", "dy", "dw"):
        assert f(**{name: None}) == NULL
    assert f(dw=A + 6 * M + 2) == ALIGN and f(dy=A + 5 * M + 1) == ALIGN and f(weights=A + 2 * M + 2) == ALIGN
    assert f(dy=A + M) == ALIAS and f(dw=A + 5 * M + 5118) == ALIGN and f(dw=A + 5 * M + 5116) == ALIAS
    assert f(dw=A + 2 * M) == ALIAS and f(dy=A + 6 * M + 158) == ALIAS


def test_quant_w4_rejections(bq_lib):
    def f(x=A, type=BF16, n=32, k=256, ld_x=256, group=64, q=A + M, ld_q=128, s=A + 2 * M, s_type=F32, ld_s=4):
        return bq_lib.bq_quant_w4(x, type, n, k, ld_x, group, q, ld_q, s, s_type, ld_s, None)
    assert f(n=0, x=None) == OK and f(k=0, q=None) == OK
    assert f(type=5) == SHAPE and f(s_type=-1) == SHAPE and f(group=48) == SHAPE and f(k=288, ld_x=288) == SHAPE
    assert f(n=-1) == SHAPE and f(ld_x=255) == SHAPE and f(ld_q=127) == SHAPE and f(ld_s=3) == SHAPE
    for name in ("x", "q", "s"):
        assert f(**{name: None}) == NULL
    assert f(x=A + 8) == ALIGN and f(ld_x=260) == ALIGN and f(q=A + M + 4) == ALIGN and f(ld_q=136) == ALIGN
    assert f(s=A + 2 * M + 2) == ALIGN
    assert f(q=A + 16) == ALIAS and f(s=A + M + 4092) == ALIAS and f(s=A) == ALIAS


def test_matvec_w4_rejections(bq_lib):
    def f(x=A, type=BF16, rows=4, k=256, ld_x=256, q=A + M, n=32, ld_q=128, s=A + 2 * M, s_type=BF16, group=64, ld_s=4,
          out=A + 3 * M, ld_out=32):
        return bq_lib.bq_matvec_w4(x, type, rows, k, ld_x, q, n, ld_q, s, s_type, group, ld_s, out, ld_out, None)
    assert f(rows=0, x=None) == OK and f(n=0, out=None) == OK
    assert f(type=F32) == SHAPE and f(s_type=F16) == SHAPE and f(type=F16) == SHAPE  # scales of the other 16-bit type
    assert f(group=16) == SHAPE and f(group=96) == SHAPE and f(k=288, ld_x=288, ld_q=144, ld_s=5) == SHAPE
    assert f(k=-64) == SHAPE and f(rows=-1) == SHAPE and f(n=-1) == SHAPE
    assert f(n=2 ** 24 + 1) == SHAPE and f(rows=2 ** 31) == SHAPE
    assert f(ld_x=248) == SHAPE and f(ld_q=112) == SHAPE and f(ld_s=3) == SHAPE and f(ld_out=31) == SHAPE
    for name in ("x", "q", "s", "out"):
        assert f(**{name: None}) == NULL
    assert f(x=A + 8) == ALIGN and f(ld_x=260) == ALIGN and f(q=A + M + 8) == ALIGN and f(ld_q=136) == ALIGN
    assert f(s=A + 2 * M + 2) == ALIGN and f(out=A + 3 * M + 1) == ALIGN
    assert f(out=A + 2046) == ALIAS and f(out=A + M + 4094) == ALIAS and f(out=A + 2 * M + 254) == ALIAS


def test_matvec_w4_experts_rejections(bq_lib):
    def f(x=A, type=F16, x_rows=10, k=256, ld_x=256, q=A + M, n=32, ld_q=128, eq=4096, s=A + 2 * M, s_type=F32,
          group=128, ld_s=2, es=64, offsets=A + 3 * M, experts=8, order=A + 4 * M, top_k=4, slots=40, out=A + 5 * M,
          ld_out=32):
        return bq_lib.bq_matvec_w4_experts(x, type, x_rows, k, ld_x, q, n, ld_q, eq, s, s_type, group, ld_s, es,
                                           offsets, experts, order, top_k, slots, out, ld_out, None)
    assert f(slots=0, offsets=None, x=None) == OK
    assert f(experts=0) == SHAPE and f(experts=1025) == SHAPE and f(top_k=0) == SHAPE and f(top_k=65) == SHAPE
    assert f(x_rows=9) == SHAPE and f(order=None) == SHAPE  # fewer rows than the places need
    assert f(eq=4080) == SHAPE and f(es=63) == SHAPE and f(slots=-1) == SHAPE
    for name in ("x", "q", "s", "offsets", "out"):
        assert f(**{name: None}) == NULL
    assert f(eq=4104) == ALIGN and f(offsets=A + 3 * M + 2) == ALIGN and f(order=A + 4 * M + 1) == ALIGN
    assert f(out=A + M + 8 * 4096 - 2) == ALIAS and f(out=A + 3 * M + 34) == ALIAS and f(out=A + 4 * M) == ALIAS


def test_the_binding_refuses_other_devices(bq_lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    plan = experts.empty_plan(4, 2, 8, device="cpu")
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="ids is on the CPU"):
        experts.sort(torch.zeros((4, 2), dtype=torch.int64), 8, *plan)
    with pytest.raises(ValueError, match="x is on the CPU"):
        experts.gather(x, plan.inverse, plan.offsets, x)
    with pytest.raises(ValueError, match="y is on the CPU"):
        experts.combine(x, None, plan.inverse, x)
    with pytest.raises(ValueError, match="dout is on the CPU"):
        experts.combine_grad(x, x, x, plan.inverse, plan.offsets, x, x)
    with pytest.raises(ValueError, match="x is on the CPU"):
        w4.matvec_w4(x, x, x, x)
    with pytest.raises(ValueError, match="x is on the CPU"):
        w4.matvec_w4_experts(x, x, x, plan.offsets, x)


@pytest.fixture
def on_device(monkeypatch):
    """CPU tensors pass for CUDA tensors, and a call that reaches the library fails."""
    class Closed:
        def __getattr__(self, name):
            return lambda *args: pytest.fail(f"{name} was called")
    for module in (experts, w4):
        monkeypatch.setattr(module, "_here", lambda *args: 0)
        monkeypatch.setattr(module, "_on", lambda *args: 0)
        monkeypatch.setattr(module, "load", lambda: Closed())


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_the_binding_checks_shapes_and_types(on_device):
    plan = experts.empty_plan(4, 2, 8, device="cpu")
    ids, x, y, w = z(4, 2, dtype=torch.int64), z(4, 64), z(8, 64), z(4, 2, dtype=torch.float32)
    with pytest.raises(ValueError, match="tokens, top_k"):
        experts.sort(ids[0], 8, *plan)
    with pytest.raises(ValueError, match="offsets must have"):
        experts.sort(ids, 9, *plan)
    with pytest.raises(ValueError, match="workspace"):
        experts.sort(ids, 8, *plan[:3], plan.workspace[:100])
    for bad in (ids.float(), ids.short()):
        with pytest.raises(TypeError, match="ids: expected"):
            experts.sort(bad, 8, *plan)
    with pytest.raises(ValueError, match=r"out: expected shape \(8, 64\)"):
        experts.gather(x, plan.inverse, plan.offsets, z(4, 64))
    with pytest.raises(TypeError, match="x: expected bfloat16"):
        experts.gather(z(4, 64, dtype=torch.float64), plan.inverse, plan.offsets, y)
    with pytest.raises(TypeError, match="out: expected"):
        experts.gather(x, plan.inverse, plan.offsets, y.half())
    with pytest.raises(ValueError, match="unit column stride"):
        experts.gather(z(64, 4).T, plan.inverse, plan.offsets, y)
    with pytest.raises(ValueError, match="weights must be"):
        experts.combine(y, w[:3], plan.inverse, x)
    with pytest.raises(ValueError, match="weights and dweights"):
        experts.combine_grad(x, y, w, plan.inverse, plan.offsets, y, w[:3])


def test_the_binding_checks_weights(on_device):
    u8 = dict(dtype=torch.uint8)
    x, q, s, out = z(3, 256), z(16, 128, **u8), z(16, 4), z(3, 16)
    with pytest.raises(TypeError, match="q must be uint8"):
        w4.matvec_w4(x, q.char(), s, out)
    with pytest.raises(TypeError, match="x must be"):
        w4.matvec_w4(x.float(), q, s, out)
    with pytest.raises(TypeError, match="scales must be"):
        w4.matvec_w4(x, q, s.half(), out)
    with pytest.raises(ValueError, match="x must be"):
        w4.matvec_w4(z(3, 128), q, s, out)
    for groups in (1, 3, 16):
        with pytest.raises(ValueError, match="a scale covers"):
            w4.matvec_w4(x, q, z(16, groups), out)
    with pytest.raises(ValueError, match="alike but the last"):
        w4.matvec_w4(x, q, z(15, 4), out)
    with pytest.raises(ValueError, match="out: expected shape"):
        w4.matvec_w4(x, q, s, z(3, 15))
    qe, se = z(5, 16, 128, **u8), z(5, 16, 4)
    offsets = z(6, dtype=torch.int32)
    with pytest.raises(ValueError, match="offsets must have"):
        w4.matvec_w4_experts(x, qe, se, offsets[:5], out)
    with pytest.raises(ValueError, match="order must have"):
        w4.matvec_w4_experts(x, qe, se, offsets, out, order=z(2, dtype=torch.int32))


def test_a_product_over_no_columns_reaches_the_launch(bq_lib):
    # in a process of its own that sees no GPU: the call passes every check and fails at the launch
    calls = """
import sys
from block_quantized_wire_gb300 import _lib
lib, A, M = _lib.load(), 0x7F0000000000, 0x1000000
for rows in (1, 3, 40):
    assert lib.bq_matvec_w4(None, 0, rows, 0, 0, None, 24000, 0, None, 0, 32, 0, A, 24000, None) == 5
    assert lib.bq_matvec_w4_experts(None, 0, rows, 0, 0, None, 24000, 0, 0, None, 0, 32, 0, 0, A + M, 8, None, 1, rows,
                                    A + 2 * M, 24000, None) == 5
"""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", calls], capture_output=True, text=True, env=env, cwd=build.ROOT)
    assert r.returncode == 0, (r.returncode, r.stderr)
