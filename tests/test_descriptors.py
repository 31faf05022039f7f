"""The cache descriptors keep their C struct between calls: what it says follows the fields."""
from __future__ import annotations

import copy
import pickle

import pytest
import torch


@pytest.fixture(scope="module")
def pkm():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_mla_gb300
    return paged_kv_mla_gb300


def make(pkm, quantised):
    sizes = dict(page_table=torch.zeros(2, 4, dtype=torch.int32), layer_stride=64, page_stride=32,
                 slot_stride=16, num_layers=1, num_pages=2, page_size=2)
    if quantised:
        return pkm.QuantCache(data=torch.zeros(64, dtype=torch.uint8), kv_lora_rank=128, rope_dim=8, **sizes)
    return pkm.PagedCache(data=torch.zeros(64, dtype=torch.int16), row_elems=16, **sizes)


@pytest.mark.parametrize("quantised", [False, True])
def test_struct_follows_the_fields(pkm, quantised):
    c = make(pkm, quantised)
    s = c.c_struct()
    assert c.c_struct() is s and s.page_size == 2 and s.cache_lengths is None
    c.page_size = 4
    assert c.c_struct().page_size == 4
    c.cache_lengths = torch.zeros(2, dtype=torch.int32)
    assert c.c_struct().cache_lengths == c.cache_lengths.data_ptr()
    s = c.c_struct()
    c.data.set_(torch.zeros(128, dtype=c.data.dtype))   # other memory behind the same tensor
    c.page_table.set_(torch.zeros(2, 6, dtype=torch.int32))
    assert c.c_struct() is s
    assert s.data == c.data.data_ptr() and s.page_table == c.page_table.data_ptr()
    assert s.max_pages_per_seq == 6


@pytest.mark.parametrize("quantised", [False, True])
def test_copies_are_their_own(pkm, quantised):
    c = make(pkm, quantised)
    c.c_struct()
    for d in (copy.copy(c), copy.deepcopy(c), pickle.loads(pickle.dumps(c))):
        d.page_size = 8
        assert d.c_struct().page_size == 8 and c.c_struct().page_size == 2
