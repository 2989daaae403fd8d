"""The 4-bit cache without a GPU: the C ABI's refusals (before any CUDA call; the fake pointers are
never dereferenced), the binding's checks of tensors, and the slots of positions."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from block_quantized_wire_gb300 import build, experts, kv4
from block_quantized_wire_gb300._lib import Kv4Cache

OK, NULL, SHAPE, ALIGN, ALIAS = range(5)
A = 0x7F0000000000  # a 256-byte-aligned fake device address
M = 0x10000000
BF16, F16, F32 = range(3)


def cache_of(**more):
    """100 pages of 16 tokens, 4 heads of 128 in groups of 64: [pages][heads][page]."""
    f = dict(k=A, v=A + M, k_scales=A + 2 * M, v_scales=A + 3 * M, pages=100, heads=4, page=16, head_dim=128, group=64,
             type=BF16, page_stride=4096, head_stride=1024, token_stride=64, page_stride_s=512, head_stride_s=128,
             token_stride_s=8)
    return Kv4Cache(**(f | more))


def write(lib, rk=A + 4 * M, k_token=512, k_head=128, rv=A + 5 * M, v_token=512, v_head=128, tokens=10, slots=A + 6 * M,
          wide=1, cache=None, **more):
    c = cache_of(**more) if cache is None else cache
    return lib.bq_kv4_write(ctypes.byref(c), rk, k_token, k_head, rv, v_token, v_head, tokens, slots, wide, None)


def read(lib, rk=A + 4 * M, k_token=512, k_head=128, rv=A + 5 * M, v_token=512, v_head=128, tokens=10, slots=A + 6 * M,
         wide=1, **more):
    c = cache_of(**more)
    return lib.bq_kv4_read(ctypes.byref(c), slots, wide, tokens, rk, k_token, k_head, rv, v_token, v_head, None)


def attend(lib, q=A + 4 * M, q_ld=(1024, 1024, 128), batch=3, n_q=1, q_heads=8, table=A + 5 * M, ld_table=20, width=20,
           lengths=A + 6 * M, scale=0.1, window=0, out=A + 7 * M, out_ld=(1024, 1024, 128), lse=A + 8 * M,
           ws=A + 9 * M, ws_bytes=1 << 27, **more):
    c = cache_of(**more)
    return lib.bq_kv4_attend(ctypes.byref(c), q, *q_ld, batch, n_q, q_heads, table, ld_table, width, lengths, scale,
                             window, out, *out_ld, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [write, read, attend])
def test_cache_rejections(bq_lib, call):
    def f(**more):
        return call(bq_lib, **more)
    assert f(type=F32) == SHAPE and f(type=-1) == SHAPE
    for dim in (0, 32, 96, 320):
        assert f(head_dim=dim) == SHAPE
    assert f(group=16) == SHAPE and f(group=256) == SHAPE and f(head_dim=192, group=128) == SHAPE
    assert f(pages=-1) == SHAPE and f(pages=2 ** 31) == SHAPE and f(heads=0) == SHAPE and f(heads=1025) == SHAPE
    assert f(page=0) == SHAPE and f(page=65537) == SHAPE
    # rows that overlap: in any order of the strides
    assert f(token_stride=48) == SHAPE and f(head_stride=1008) == SHAPE and f(page_stride=4080) == SHAPE
    assert f(token_stride=-64) == SHAPE and f(head_stride=0) == SHAPE and f(page_stride_s=504) == SHAPE
    assert f(token_stride=256, head_stride=64, page_stride=4080) == SHAPE
    assert f(token_stride=2 ** 31 // 15 // 16 * 16 + 16, page_stride=2 ** 40, head_stride=64) == SHAPE  # past 2^31 in a page
    for name, base in (("k", 0), ("v", 1), ("k_scales", 2), ("v_scales", 3)):
        assert f(**{name: None}) == NULL
        assert f(**{name: A + base * M + 4}) == ALIGN
    assert f(token_stride=72, head_stride=1152, page_stride=4608) == ALIGN and f(head_stride=1032, page_stride=4128) == ALIGN
    assert f(token_stride_s=12, head_stride_s=192, page_stride_s=768) == ALIGN  # pairs of 8 bytes a row
    assert f(v=A + 99 * 4096 + 4080) == ALIAS and f(k_scales=A + M + 512) == ALIAS
    assert f(v_scales=A + 2 * M + 99 * 512 + 504) == ALIAS


def test_a_cache_may_keep_all_arrays_of_a_page_in_one_block(bq_lib):
    # keys, values and their pairs of each page, one after the other; nothing is launched for no tokens
    block = dict(v=A + 4096, k_scales=A + 8192, v_scales=A + 8192 + 512, page_stride=9216, page_stride_s=9216)
    assert write(bq_lib, tokens=0, **block) == OK
    assert write(bq_lib, tokens=0, **(block | dict(v=A + 4080))) == ALIAS
    assert write(bq_lib, tokens=0, **(block | dict(v_scales=A + 8192 + 504))) == ALIAS
    assert write(bq_lib, tokens=0, **(block | dict(v_scales=A + 9216 - 504))) == ALIAS  # past its page
    assert write(bq_lib, tokens=0, **(block | dict(page_stride_s=9232))) == ALIAS  # pages that drift


@pytest.mark.parametrize("call", [write, read])
def test_rows_rejections(bq_lib, call):
    def f(**more):
        return call(bq_lib, **more)
    assert f(tokens=0, rk=None, rv=None, slots=None) == OK
    assert f(tokens=-1) == SHAPE and f(tokens=2 ** 25) == SHAPE  # 2^34 values
    assert f(k_token=-512) == SHAPE and f(v_head=-128) == SHAPE
    for name in ("rk", "rv", "slots"):
        assert f(**{name: None}) == NULL
    assert f(rk=A + 4 * M + 8) == ALIGN and f(k_token=516) == ALIGN and f(v_head=132, v_token=1024) == ALIGN
    assert f(slots=A + 6 * M + 4) == ALIGN and f(slots=A + 6 * M + 2, wide=0) == ALIGN
    assert f(rk=A + 4096) == ALIAS and f(rv=A + 2 * M) == ALIAS and f(rv=A + 3 * M + 99 * 512 + 496) == ALIAS


def test_rows_that_are_written_are_apart(bq_lib):
    assert read(bq_lib, k_token=504) == SHAPE and read(bq_lib, v_head=120) == SHAPE and read(bq_lib, k_token=0) == SHAPE
    assert read(bq_lib, rv=A + 4 * M + 4096) == ALIAS and read(bq_lib, slots=A + 4 * M) == ALIAS
    assert write(bq_lib, slots=A + 64) == ALIAS


def test_attend_rejections(bq_lib):
    def f(**more):
        return attend(bq_lib, **more)
    assert f(batch=0, q=None) == OK and f(n_q=0, out=None) == OK and f(q_heads=0, table=None) == OK
    assert f(batch=-1) == SHAPE and f(n_q=-1) == SHAPE and f(q_heads=6) == SHAPE and f(q_heads=-4) == SHAPE
    assert f(q_heads=65540) == SHAPE and f(n_q=131073, q_heads=8) == SHAPE
    assert f(width=-1) == SHAPE and f(width=2 ** 27, ld_table=2 ** 27) == SHAPE and f(ld_table=19) == SHAPE
    assert f(window=-1) == SHAPE and f(window=2 ** 30 + 1) == SHAPE
    assert f(scale=float("nan")) == SHAPE and f(scale=float("inf")) == SHAPE
    assert f(out_ld=(1016, 1024, 128)) == SHAPE and f(out_ld=(1024, 1024, 120)) == SHAPE and f(q_ld=(-8, 0, 128)) == SHAPE
    need = bq_lib.bq_kv4_workspace_bytes(4, 128, 1, 8)
    assert need >= 0 and f(ws_bytes=need - 1) == SHAPE
    for name in ("q", "table", "lengths", "out", "ws"):
        assert f(**{name: None}) == NULL
    assert f(q=A + 4 * M + 8) == ALIGN and f(q_ld=(1028, 1024, 128)) == ALIGN and f(out=A + 7 * M + 2) == ALIGN
    assert f(table=A + 5 * M + 2) == ALIGN and f(lengths=A + 6 * M + 1) == ALIGN and f(lse=A + 8 * M + 2) == ALIGN
    assert f(ws=A + 9 * M + 8) == ALIGN
    assert f(out=A + 4 * M) == ALIAS and f(out=A + 5 * M) == ALIAS and f(out=A) == ALIAS
    assert f(lse=A + 7 * M) == ALIAS and f(lse=A + 6 * M) == ALIAS
    if need > 0:
        assert f(out=A + 9 * M) == ALIAS and f(ws=A + 3 * M + 512) == ALIAS and f(ws=A + 4 * M) == ALIAS


def test_workspace_of_refused_shapes(bq_lib):
    f = bq_lib.bq_kv4_workspace_bytes
    for bad in ((0, 128, 1, 8), (1025, 128, 1, 1025), (4, 96, 1, 8), (4, 128, 0, 8), (4, 128, 1, 6), (4, 128, 2 ** 18, 8)):
        assert f(*bad) == -1
    for dim in (64, 128, 192, 256):
        assert f(8, dim, 1, 64) >= 0


def test_valid_calls_reach_the_launch(bq_lib):
    # in a process of its own that sees no GPU: the calls pass every check and fail at the launch
    calls = """
from tests.test_kv4_host import *
from block_quantized_wire_gb300 import _lib
lib = _lib.load()
block = dict(v=A + 4096, k_scales=A + 8192, v_scales=A + 8192 + 512, page_stride=9216, page_stride_s=9216)
for call in (write, read, attend):
    assert call(lib) == 5 and call(lib, **block) == 5
    assert call(lib, token_stride=256, head_stride=64, token_stride_s=32, head_stride_s=8) == 5
    assert call(lib, pages=0, k=None, v=None, k_scales=None, v_scales=None) == 5
    assert call(lib, pages=1, page_stride=-1, page_stride_s=3) == 5  # no second page to step to
assert write(lib, k_token=0, v_head=0) == 5  # a row given to every token, or to every head
assert attend(lib, width=0, ld_table=0, table=None) == 5 and attend(lib, lse=None, n_q=3, out_ld=(4096, 1024, 128)) == 5
assert attend(lib, scale=-1.0, window=2 ** 30, batch=1, ld_table=0) == 5
"""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", calls], capture_output=True, text=True, env=env, cwd=build.ROOT)
    assert r.returncode == 0, (r.returncode, r.stderr)


@pytest.fixture
def on_device(monkeypatch):
    """CPU tensors pass for CUDA tensors, and a call that reaches the library fails."""
    class Closed:
        def __getattr__(self, name):
            return lambda *args: pytest.fail(f"{name} was called")
    monkeypatch.setattr(kv4, "_here", lambda *args: 0)
    monkeypatch.setattr(kv4, "_on", lambda *args: 0)
    monkeypatch.setattr(kv4, "load", lambda: Closed())


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def parts(pages=6, heads=2, page=8, dim=64, group=32, dtype=torch.bfloat16):
    codes, pairs = (pages, heads, page, dim // 2), (pages, heads, page, dim // group, 2)
    return [z(*codes, dtype=torch.uint8), z(*pairs, dtype=dtype), z(*codes, dtype=torch.uint8), z(*pairs, dtype=dtype)]


def test_the_binding_refuses_other_devices(bq_lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    cache = kv4.Cache(*parts())
    rows = z(3, 2, 64)
    with pytest.raises(ValueError, match="k is on the CPU"):
        kv4.write(rows, rows, z(3, dtype=torch.int64), cache)
    with pytest.raises(ValueError, match="cache is on the CPU"):
        kv4.read(cache, z(3, dtype=torch.int64), rows, rows)
    with pytest.raises(ValueError, match="q is on the CPU"):
        kv4.attend(z(1, 1, 2, 64), cache, z(1, 1, dtype=torch.int32), z(1, dtype=torch.int32), z(1, 1, 2, 64), rows)


def test_the_cache_checks_its_tensors():
    k, ks, v, vs = parts()
    kv4.Cache(k, ks, v, vs)
    kv4.Cache(*(t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, ks, v, vs)))  # tokens before heads
    with pytest.raises(TypeError, match="codes must be uint8"):
        kv4.Cache(k.char(), ks, v, vs)
    for bad in (ks.float(), ks.half()):
        with pytest.raises(TypeError, match="scales must be"):
            kv4.Cache(k, ks, v, bad)
    with pytest.raises(TypeError, match="scales must be"):
        kv4.Cache(k, ks.float(), v, vs.float())
    with pytest.raises(ValueError, match="codes must be"):
        kv4.Cache(k, ks[..., 0], v, vs)
    with pytest.raises(ValueError, match="codes must be"):
        kv4.Cache(k[:5], ks, v, vs)
    with pytest.raises(ValueError, match="same shapes"):
        kv4.Cache(k, ks, v[:, :, :7], vs)
    for dim, groups in ((96, 3), (128, 8), (64, 3), (320, 5)):
        bad = [z(2, 1, 4, dim // 2, dtype=torch.uint8), z(2, 1, 4, groups, 2)] * 2
        with pytest.raises(ValueError, match="head_dim must be"):
            kv4.Cache(*bad)
    with pytest.raises(ValueError, match="must be contiguous"):
        kv4.Cache(k.transpose(2, 3).contiguous().transpose(2, 3), ks, v, vs)
    with pytest.raises(ValueError, match="same strides"):
        kv4.Cache(k, ks, v.transpose(1, 2).contiguous().transpose(1, 2), vs)
    with pytest.raises(ValueError, match="a scale covers"):
        kv4.empty_cache(4, 1, 16, 192, group=128, device="cpu")
    assert kv4.empty_cache(4, 1, 16, 64, group=64, device="cpu").k_scales.shape == (4, 1, 16, 1, 2)


def test_the_binding_checks_rows(on_device):
    cache = kv4.Cache(*parts())
    rows, at = z(3, 2, 64), z(3, dtype=torch.int32)
    for call in (lambda k, v, s: kv4.write(k, v, s, cache), lambda k, v, s: kv4.read(cache, s, k, v)):
        with pytest.raises(TypeError, match="k must be torch.bfloat16"):
            call(rows.half(), rows, at)
        with pytest.raises(ValueError, match=r"v must be \[3, 2, 64\]"):
            call(rows, rows[:2], at)
        with pytest.raises(ValueError, match=r"k must be \[4, 2, 64\]"):
            call(rows, rows, z(4, dtype=torch.int32))
        with pytest.raises(ValueError, match="unit column stride"):
            call(rows, z(3, 64, 2).transpose(1, 2), at)
        with pytest.raises(ValueError, match="one dimension"):
            call(rows, rows, at[None])
        with pytest.raises(TypeError, match="slots: expected"):
            call(rows, rows, at.short())
        with pytest.raises(ValueError, match="contiguous"):
            call(rows, rows, z(6, dtype=torch.int32)[::2])


def test_the_binding_checks_attention(on_device):
    cache = kv4.Cache(*parts())
    i32 = dict(dtype=torch.int32)
    q, table, lengths, ws = z(3, 2, 4, 64), z(3, 5, **i32), z(3, **i32), z(64, dtype=torch.uint8)

    def call(q=q, table=table, lengths=lengths, out=None, ws=ws, **more):
        kv4.attend(q, cache, table, lengths, torch.zeros_like(q) if out is None else out, ws, **more)
    with pytest.raises(TypeError, match="q must be torch.bfloat16"):
        call(q=q.half())
    for bad in (q[0], z(3, 2, 3, 64), z(3, 2, 4, 128)):
        with pytest.raises(ValueError, match="q must be"):
            call(q=bad)
    for bad in (q[:2], q.half()):
        with pytest.raises(ValueError, match="out must be"):
            call(out=bad)
    with pytest.raises(ValueError, match="unit column stride"):
        call(q=z(3, 2, 64, 4).transpose(2, 3))
    for bad in (table.long(), table[:2], table[0]):
        with pytest.raises(ValueError, match="table must be"):
            call(table=bad)
    with pytest.raises(ValueError, match="table must have unit"):
        call(table=z(5, 3, **i32).T)
    with pytest.raises(ValueError, match="lengths must be"):
        call(lengths=lengths[:2])
    with pytest.raises(TypeError, match="lengths: expected"):
        call(lengths=lengths.long())
    with pytest.raises(ValueError, match="lse must be"):
        call(lse=z(3, 2, 2, dtype=torch.float32))
    with pytest.raises(TypeError, match="lse: expected"):
        call(lse=z(3, 2, 4))
    with pytest.raises(ValueError, match="contiguous workspace"):
        call(ws=z(64, 2, dtype=torch.uint8)[:, 0])


def test_slots_of_positions():
    table = torch.tensor([[5, 2, -1], [7, 0, 3]], dtype=torch.int32)
    got = kv4.slots(table, torch.tensor([[0, 15, 16, 31, 32], [47, 48, -1, 17, 2]]), 16)
    assert got.tolist() == [[80, 95, 32, 47, -1], [63, -1, -1, 1, 114]] and got.dtype == torch.int64
    assert kv4.slots(table[:, :0], torch.zeros((2, 1), dtype=torch.int32), 16).tolist() == [[-1], [-1]]
