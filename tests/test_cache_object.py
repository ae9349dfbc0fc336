"""A KVCache is what it was made of: its descriptor holds the addresses of its tensors, so none of its fields can be replaced
(the freed memory of the old tensor would be written and read)."""
import copy

import pytest
import torch

import bit_floating_point_amd as F


def make(grid=F.grid_minifloat(4, 3)):
    return F.kv_cache(6, 2, 16, 128, grid, device="cpu")


@pytest.mark.parametrize("grid", [F.grid_minifloat(4, 3), None])
def test_fields_stay(grid):
    c = make(grid)
    for name in F.KVCache.__slots__:
        before = getattr(c, name)
        with pytest.raises(AttributeError, match="new KVCache"):
            setattr(c, name, copy.copy(before) if name != "desc" else None)
        with pytest.raises(AttributeError, match="new KVCache"):
            delattr(c, name)
        assert getattr(c, name) is before
    with pytest.raises(AttributeError):
        c.other = 1
    with pytest.raises(AttributeError, match="new KVCache"):
        c.__init__(torch.zeros(6, 2, 16, 128, dtype=torch.bfloat16), torch.zeros(6, 2, 16, 128, dtype=torch.bfloat16))
    assert c.desc.k == c.k.data_ptr() and c.desc.v == c.v.data_ptr()


def test_contents_change_and_copies_share():
    """The tensors' contents are the caller's; a copy of the object is the same cache."""
    c = make()
    c.k.fill_(3)
    c.k[0] += 1
    d = copy.copy(c)
    assert d.k is c.k and d.desc.k == c.k.data_ptr() and d.page_size == 16
