"""The attention layer's composition without a GPU: which ranks' parts are summed, and the shapes that its operators get."""
import pytest

from block_quantized_wire_gb300 import attention


@pytest.mark.parametrize("ranks,caches", [(3, 2), (2, 3), (1, 0), (0, 1)])
def test_every_rank_has_a_cache_of_its_own(ranks, caches, monkeypatch):
    # no part is left out: the counts are compared before any work
    monkeypatch.setattr(attention, "decode_part", lambda *args, **more: pytest.fail("a part was computed"))
    with pytest.raises(ValueError, match=f"{ranks} ranks.*{caches} caches"):
        attention.decode_layer(None, [None] * ranks, [None] * caches, None, None, "")
