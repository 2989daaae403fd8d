"""The attention layer's forms that a server meets: no requests, several tokens a request, a window, FP16, an own workspace,
sequences that fill their table, every kind of wire mode. The layer of test_gpu_kv4 is what is compared with."""
import pytest
import torch

from block_quantized_wire_gb300 import attention, kv4
from tests.test_gpu_kv4 import a_layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", ["", "i8_a2a", "mx_ring", "i8_ag"])
@pytest.mark.parametrize("queries", [1, 3])
def test_a_step_of_no_requests(mode, queries):
    ranks, caches, table, lengths, (x,) = a_layer(mode, steps=1)
    before = [t.clone() for c in caches for t in (c.k, c.v)]
    outs = attention.decode_layer(x[:0], ranks, caches, table[:0], lengths[:0], mode, queries=queries)
    assert all(o.numel() == 0 and o.dtype is x.dtype for o in outs)
    assert all(torch.equal(a, b) for a, b in zip(before, [t for c in caches for t in (c.k, c.v)]))
