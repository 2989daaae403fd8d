"""The attention layer's composition without a GPU: which ranks' parts are summed, and the shapes that its operators get."""
import pytest
import torch

from block_quantized_wire_gb300 import attention, kv4, w4


@pytest.mark.parametrize("ranks,caches", [(3, 2), (2, 3), (1, 0), (0, 1)])
def test_every_rank_has_a_cache_of_its_own(ranks, caches, monkeypatch):
    # no part is left out: the counts are compared before any work
    monkeypatch.setattr(attention, "decode_part", lambda *args, **more: pytest.fail("a part was computed"))
    with pytest.raises(ValueError, match=f"{ranks} ranks.*{caches} caches"):
        attention.decode_layer(None, [None] * ranks, [None] * caches, None, None, "")


@pytest.mark.parametrize("batch,queries", [(0, 1), (0, 3), (2, 3)])
def test_a_part_of_any_batch_an_empty_one_too(batch, queries, monkeypatch):
    # the operators are replaced by ones that note the shapes they are given
    seen = {}
    w = attention.HeadWeights(4, 2, (torch.zeros(8 * 64, 32, dtype=torch.uint8), None),
                              (torch.zeros(64, 128, dtype=torch.uint8), None))
    monkeypatch.setattr(w4, "matvec_w4", lambda x, q, s, out: seen.setdefault("products", []).append(
        (tuple(x.shape), tuple(out.shape))))
    monkeypatch.setattr(kv4, "write", lambda k, v, slots, cache: seen.update(
        rows=(tuple(k.shape), tuple(v.shape)), slots=slots.tolist()))
    monkeypatch.setattr(kv4, "attend", lambda q, cache, table, lengths, out, workspace, window: seen.update(
        q=tuple(q.shape), out=tuple(out.shape), window=window))
    monkeypatch.setattr(kv4, "empty_workspace", lambda q, cache: None)
    cache = kv4.empty_cache(6, 2, 16, 64, 32, device="cpu")
    table = torch.arange(3 * batch, dtype=torch.int32).view(batch, 3)
    lengths = torch.tensor([17, 2][:batch], dtype=torch.int32)
    n = batch * queries
    out = attention.decode_part(torch.zeros(n, 64, dtype=torch.bfloat16), w, cache, table, lengths, queries, window=9)
    assert out.shape == (n, 64) and seen["q"] == seen["out"] == (batch, queries, 4, 64) and seen["window"] == 9
    assert seen["rows"] == ((n, 2, 64), (n, 2, 64)) and seen["products"] == [((n, 64), (n, 512)), ((n, 256), (n, 64))]
    assert seen["slots"] == ([14, 15, 16, -1, 48, 49] if batch else [])


@pytest.mark.parametrize("heads,page", [(0, 4), (4, 0), (1025, 1), (1, 65537), (2 ** 32 + 1, 1), (1, 2 ** 32 + 16)])
def test_a_cache_past_the_librarys_sizes_is_refused(heads, page):
    # not taken as the low 32 bits of its size
    def parts(*last, dtype):
        return torch.zeros(last, dtype=dtype).expand(2, heads, page, *last)
    k, s = parts(32, dtype=torch.uint8), parts(2, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="1 to 1024 heads and 1 to 65536 tokens a page"):
        kv4.Cache(k, s, k, s)


def test_more_query_rows_than_a_call_takes_are_refused(monkeypatch):
    cache = kv4.empty_cache(2, 1, 16, 64, device="cpu")
    monkeypatch.setattr(kv4, "_here", lambda *args: 0)
    monkeypatch.setattr(kv4, "load", lambda: pytest.fail("the library was called"))
    one = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    for n_q, q_heads in ((2 ** 20 + 1, 1), (17, 65536), (1, 65537), (2 ** 32 + 1, 1)):
        q = one.expand(1, n_q, q_heads, 64)
        with pytest.raises(ValueError, match="more than a call takes"):
            kv4.attend(q, cache, torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32), q, one)
        with pytest.raises(ValueError, match="more than a call takes"):
            kv4.empty_workspace(q, cache)
