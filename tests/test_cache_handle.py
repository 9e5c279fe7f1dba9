"""The history cache's handle without a GPU: what a made cache refuses."""
import pytest

import block_sparse_attention_kunlun_b200 as ba


@pytest.mark.parametrize("name", ["k", "v", "k_scales", "v_scales", "page_table", "status", "struct", "batch", "device"])
def test_attributes_cannot_be_replaced(name):
    """The library was told the tensors' addresses: another tensor in the place of one would leave them stale."""
    cache = ba.HistoryCache.__new__(ba.HistoryCache)
    object.__setattr__(cache, name, 1)
    with pytest.raises(AttributeError, match="for good"):
        setattr(cache, name, None)
    with pytest.raises(AttributeError, match="for good"):
        delattr(cache, name)
    assert getattr(cache, name) == 1
