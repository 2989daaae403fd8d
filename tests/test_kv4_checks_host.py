"""The tight checks of attention see the mistakes that they are for: planted in 64-bit outputs, on the CPU."""
import numpy as np
import pytest
import torch

from block_quantized_wire_gb300 import kv4
from tests.kv4_checks import BITS, check_rows, check_shares, rows_of, shares


def problem(seed, lens, heads, dim, group, page, dtype):
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    cache = kv4.empty_cache(sum(need), heads, page, dim, group, dtype, device="cpu")
    for codes, pairs in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
        codes.copy_(torch.from_numpy(rng.integers(0, 256, codes.shape, dtype=np.uint8)))
        s, z = np.exp(rng.standard_normal(pairs.shape[:-1]) * 0.2) * 0.2, rng.standard_normal(pairs.shape[:-1])
        pairs.copy_(torch.from_numpy(np.stack([s, z], -1).astype(np.float32)))
    table, order, at = np.full((len(lens), max(need)), -1, np.int32), rng.permutation(sum(need)), 0
    for b, n in enumerate(need):
        table[b, :n], at = order[at:at + n], at + n
    q = torch.from_numpy(rng.standard_normal((len(lens), 1, 2 * heads, dim)).astype(np.float32)).to(dtype)
    return q, cache, torch.from_numpy(table), torch.tensor(lens, dtype=torch.int32)


@pytest.mark.parametrize("name", list(BITS))
@pytest.mark.parametrize("lens", [[300], [2049, 1], [9000, 100]])
def test_a_lost_or_doubled_tile_shows(lens, name):
    dtype = {"bf16": torch.bfloat16, "f16": torch.float16}[name]
    q, cache, table, lengths = problem(sum(lens), lens, 1, 64, 32, 64, dtype)
    rows = list(rows_of(q, cache, table, lengths, 0.125))
    right = np.zeros(q.shape)
    for row in rows:
        right[row[0]] = row[1]
    rounded = torch.from_numpy(right).to(dtype)
    check_rows(rounded, None, rows, BITS[name])
    for first in (0, 32 * (lens[0] // 64), 32 * (lens[0] // 32) - 32):
        tile = slice(first, first + 32)
        for row in rows_of(q[:1], cache, table[:1], lengths[:1], 0.125, drop=lambda b, h, at: tile):
            for wrong in (row[1], 2 * right[row[0]] - row[1]):
                bad = rounded.clone()
                bad[row[0]] = torch.from_numpy(wrong).to(dtype)
                with pytest.raises(AssertionError):
                    check_rows(bad, None, rows, BITS[name])


@pytest.mark.parametrize("length,n_q,window,dim", [(20000, 1, 0, 64), (65000, 1, 0, 64), (1000, 4, 300, 128), (33, 1, 0, 256)])
def test_a_single_lost_position_shows(length, n_q, window, dim):
    want = shares(length, n_q, window, dim)
    as_f16 = torch.from_numpy(want).half().double().numpy()
    check_shares(as_f16, want)
    last = length - n_q  # seen by every query
    for lost in (last, last - 31, last - 32, max(0, last - 250)):
        with pytest.raises(AssertionError):
            check_shares(torch.from_numpy(shares(length, n_q, window, dim, [lost])).half().double().numpy(), want)
