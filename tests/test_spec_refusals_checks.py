"""Arguments of the speculative-decoding entry points that read or write the wrong memory: each
refused by the calls' own checks, which otherwise say that the call would go on to the GPU."""
from __future__ import annotations

import pytest
import torch

from test_spec_refusals import INVALID, UNSUPPORTED, attention, b16, i32, paged, quant

GOES_ON = 3  # PKM_ERR_CUDA: nothing was found, and nothing may be launched


@pytest.fixture()
def pkm(monkeypatch):
    """The binding with its checks alone, on host memory taken for the device's."""
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_mla_gb300 as m
    monkeypatch.setattr(m, "_here", lambda device: True)
    m._lib.pkm_checks_only(1)
    yield m
    m._lib.pkm_checks_only(0)


def compact(pkm, cache, accepted, counts, new, begin=0, count=1):
    f = pkm.mla_cache_compact_paged_qcache if isinstance(cache, pkm.QuantCache) \
        else pkm.mla_cache_compact_paged
    return f(cache, begin, count, accepted, counts, new, stream=0, check=False)


@pytest.mark.parametrize("make", [paged, quant])
def test_new_lengths_share_no_memory(pkm, make):
    """Blocks of a request's other layers still read what its first block would overwrite."""
    words = i32(64)
    acc, cnt, new = words[0:6].view(2, 3), words[6:8], words[8:10]
    lengths, table = words[10:12], words[12:20].view(2, 4)
    cache = make(pkm, cache_lengths=lengths, page_table=table)
    assert compact(pkm, cache, acc, cnt, new) == GOES_ON
    assert compact(pkm, cache, acc, cnt, None) == GOES_ON
    assert compact(pkm, cache, acc, cnt, cnt) == INVALID
    for at in range(0, 20):
        free = at == 8
        assert compact(pkm, cache, acc, cnt, words[at:at + 2]) == (GOES_ON if free else INVALID), at
    assert compact(pkm, cache, acc, cnt, words[20:22]) == GOES_ON


@pytest.mark.parametrize("make,wide", [(paged, 576), (quant, 656)])
def test_layers_that_share_rows(pkm, make, wide):
    """The threads of one layer would move what those of another have yet to read."""
    def call(count=2, **kw):
        return compact(pkm, make(pkm, num_layers=3, **kw), i32(2, 3), i32(2), i32(2), count=count)

    assert call() == GOES_ON
    assert call(layer_stride=0) == INVALID and call(layer_stride=0, count=1) == GOES_ON
    assert call(layer_stride=wide - 16) == INVALID and call(layer_stride=wide) == GOES_ON
    assert call(slot_stride=wide - 16) == INVALID


def test_planes_that_share_rows(pkm):
    def call(count=3, **kw):
        return compact(pkm, paged(pkm, num_layers=3, **kw), i32(2, 3), i32(2), i32(2), count=count)

    apart = dict(layer_stride=1152 * 64, slot_stride=1152, page_stride=1152 * 16)
    assert call(kv_stride=576, **apart) == GOES_ON
    assert call(kv_stride=568, **apart) == INVALID
    assert call(kv_stride=568, count=1, **apart) == INVALID
    for layers in (1, 2):  # the V plane on a later layer's K plane
        assert call(kv_stride=layers * 1152 * 64, **apart) == INVALID
        assert call(kv_stride=layers * 1152 * 64 - 576, **apart) == GOES_ON
        assert call(kv_stride=layers * 1152 * 64 - 568, **apart) == INVALID
        assert call(kv_stride=layers * 1152 * 64 + 568, **apart) == INVALID
        assert call(kv_stride=layers * 1152 * 64 + 576, **apart) == GOES_ON
    assert call(kv_stride=3 * 1152 * 64, **apart) == GOES_ON  # behind all
    assert call(kv_stride=1152 * 64, count=1, **apart) == GOES_ON
    assert call(page_size=1, slot_stride=0, page_stride=576) == GOES_ON


def test_heads_that_a_thread_cannot_count(pkm):
    """A head behind the last of 2^31 - 1 would get a negative number, and an address."""
    x, f, pos = torch.zeros(64, dtype=torch.int16), torch.zeros(4, 8), i32(1)

    def call(heads):
        return pkm._lib.mla_rope_heads(x.data_ptr(), 0, 0, pos.data_ptr(), 1, heads, 8, f.data_ptr(),
                                       4, 0, x.data_ptr() + 64, 8, 8, None, None)

    assert call(2 ** 31 - 513) == GOES_ON
    assert call(2 ** 31 - 512) == call(2 ** 31 - 1) == UNSUPPORTED


def attend(pkm, cache, offsets=None, **kw):
    return attention(pkm, cache, offsets=offsets, **kw)


def write(pkm, cache, latent=None, offsets=None, positions=None, gamma=None, freqs=None):
    args = (b16(3, 576) if latent is None else latent, i32(3) if offsets is None else offsets,
            i32(3) if positions is None else positions,
            torch.zeros(512) if gamma is None else gamma, 1e-6,
            torch.zeros(8, 64) if freqs is None else freqs, cache, 0)
    if isinstance(cache, pkm.QuantCache):
        return pkm.mla_cache_write_paged_qcache_at(*args, stream=0, check=False)
    return pkm.mla_cache_write_paged_at(*args, 512, 64, stream=0, check=False)


def move(pkm, cache):
    return compact(pkm, cache, i32(2, 3), i32(2), i32(2))


CALLS = pytest.mark.parametrize("call", [attend, write, move])
MAKES = pytest.mark.parametrize("make", [paged, quant])


@CALLS
@MAKES
def test_descriptors_of_fewer_requests(pkm, call, make):
    """Table rows, lengths and their types as the call's requests need them."""
    assert call(pkm, make(pkm)) == GOES_ON
    assert call(pkm, make(pkm, page_table=i32(5, 4), cache_lengths=i32(5))) == GOES_ON
    for table in (i32(1, 4), i32(8), i32(2, 4).long(), i32(2, 8)[:, :4], i32(2, 4, 1)):
        assert call(pkm, make(pkm, page_table=table)) == INVALID
    for lengths in (i32(1), i32(2).long(), i32(4)[::2], None):
        assert call(pkm, make(pkm, cache_lengths=lengths)) == INVALID


@pytest.mark.parametrize("field", ["data", "page_table", "cache_lengths"])
@CALLS
@MAKES
def test_descriptors_in_other_memory(pkm, monkeypatch, call, make, field):
    """A descriptor's tensor on another device than the rest."""
    real, devices, cache = pkm._look, [], make(pkm)

    class There:  # stands for the field's tensor
        def __init__(self, t):
            self.t = t

        def __getattr__(self, name):
            return getattr(self.t, name)

        def get_device(self):
            return 1

    def look(tensors):
        found = real(tuple((*k, There(t) if t is getattr(cache, field) else t) for *k, t in tensors))
        devices.append(found[0])
        return found

    monkeypatch.setattr(pkm, "_look", look)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(pkm, "_here", lambda device: device == 0)
    pkm._lib.pkm_checks_only(0)
    assert call(pkm, cache) == INVALID and devices == [-1]


@MAKES
@pytest.mark.parametrize("what", [
    dict(q=torch.float16), dict(out=torch.float16), dict(mask=torch.float32),
    dict(lse=torch.int32), dict(offsets=torch.float32)])
def test_attention_types(pkm, make, what):
    """Elements of the right size and the wrong type, which would be read as other values."""
    (name, dtype), = what.items()
    shapes = dict(q=(3, 2, 576), out=(3, 2, 512), mask=(3, 1), lse=(3, 2), offsets=(3,))
    right = dict(q=torch.bfloat16, out=torch.bfloat16, mask=torch.uint32, lse=torch.float32,
                 offsets=torch.uint32)

    def call(dtypes):
        t = {k: torch.zeros(shapes[k], dtype=d) for k, d in dtypes.items()}
        n = pkm.mla_tree_attention_paged_workspace_size(3, 2, 512)
        raw = torch.zeros(n + 256, dtype=torch.uint8)
        kw = dict(tree_mask=t["mask"], lse=t["lse"], stream=0, check=False)
        ws, cache = raw[-raw.data_ptr() % 256:][:n], make(pkm)
        if make is quant:
            return pkm.mla_tree_attention_paged_qcache(t["q"], t["offsets"], 1.0, cache, 0,
                                                       t["out"], ws, **kw)
        return pkm.mla_tree_attention_paged(t["q"], t["offsets"], 1.0, cache, 0, 512, 64, t["out"],
                                            ws, **kw)

    assert call(right) == GOES_ON
    assert call({**right, name: dtype}) == INVALID


def test_rope_types(pkm):
    def call(x=torch.bfloat16, y=torch.bfloat16, positions=torch.uint32, freqs=torch.float32):
        return pkm.mla_rope_heads(torch.zeros(3, 4, 16, dtype=x), torch.zeros(3, dtype=positions),
                                  torch.zeros(4, 16, dtype=freqs), torch.zeros(3, 4, 16, dtype=y),
                                  stream=0, check=False)

    assert call() == GOES_ON and call(x=torch.int16, y=torch.int16, positions=torch.int32) == GOES_ON
    assert call(x=torch.float16) == call(y=torch.float16) == INVALID
    assert call(positions=torch.float32) == call(freqs=torch.int32) == INVALID


@CALLS
@MAKES
def test_descriptor_types(pkm, call, make):
    assert call(pkm, make(pkm, page_table=torch.zeros(2, 4))) == INVALID
    assert call(pkm, make(pkm, cache_lengths=torch.zeros(2))) == INVALID


@MAKES
def test_compaction_types(pkm, make):
    for bad in range(3):
        args = [torch.zeros(s, dtype=torch.float32 if i == bad else torch.uint32)
                for i, s in enumerate([(2, 3), (2,), (2,)])]
        assert compact(pkm, make(pkm), *args) == INVALID
    assert compact(pkm, make(pkm), *(a.view(torch.uint32) for a in (i32(2, 3), i32(2), i32(2)))) == GOES_ON


@MAKES
def test_rows_to_be_written(pkm, make):
    """What the cache write at positions takes for rows, offsets and factors."""
    def call(**kw):
        return write(pkm, make(pkm), **kw)

    good = dict(latent=torch.zeros(3, 576, dtype=torch.bfloat16), offsets=i32(3).view(torch.uint32),
                positions=i32(4), gamma=torch.ones(600), freqs=torch.zeros(8, 64))
    assert call() == call(**good) == GOES_ON
    for bad in (dict(latent=b16(3, 640)), dict(latent=b16(3, 640)[:, :576]), dict(latent=b16(3 * 576)),
                dict(latent=torch.zeros(3, 576, dtype=torch.float16)),
                dict(latent=torch.zeros(3, 576)), dict(offsets=i32(3).long()), dict(offsets=i32(6)[::2]),
                dict(positions=i32(2)), dict(positions=i32(3).long()), dict(gamma=torch.ones(511)),
                dict(gamma=torch.ones(512).bfloat16()), dict(gamma=torch.ones(1024)[::2]),
                dict(freqs=torch.zeros(8, 32)), dict(freqs=torch.zeros(8, 64).bfloat16()),
                dict(freqs=torch.zeros(8, 128)[:, :64]), dict(freqs=torch.zeros(512))):
        assert call(**{**good, **bad}) == INVALID, bad.keys()


def test_rows_without_rope_columns(pkm):
    cache = paged(pkm, cols=512)
    for freqs in (torch.zeros(8, 0), torch.zeros(8, 64), torch.zeros(8)):
        assert pkm.mla_cache_write_paged_at(b16(3, 512), i32(3), i32(3), torch.ones(512), 1e-6, freqs,
                                            cache, 0, 512, 0, stream=0, check=False) == GOES_ON


def test_rope_table_has_a_row_a_position(pkm):
    """Of a table in another form the rows that there are would be counted wrongly."""
    x = b16(3, 4, 16)

    def call(f):
        return pkm.mla_rope_heads(x, i32(3), f, b16(3, 4, 16), stream=0, check=False)

    assert call(torch.zeros(4, 16)) == GOES_ON
    for f in (torch.zeros(16), torch.zeros(4, 2, 16), torch.zeros(4, 8, 2), torch.zeros(4, 32)):
        assert call(f) == INVALID


@MAKES
def test_tensors_without_dimensions(pkm, make):
    """Refused like other shapes, not by an error of the binding."""
    none = torch.zeros((), dtype=torch.int32)
    assert compact(pkm, make(pkm), none, i32(2), i32(2)) == INVALID
    assert write(pkm, make(pkm), latent=torch.zeros((), dtype=torch.int16)) == INVALID
    assert attend(pkm, make(pkm), q=torch.zeros((), dtype=torch.int16), mask=i32(3, 1)) == INVALID


@pytest.mark.parametrize("kw", [dict(num_pages=2 ** 31 - 1, page_stride=1 << 33),
                                dict(num_pages=1 << 30, page_stride=1 << 35),
                                dict(page_size=(1 << 30) + 4, slot_stride=1 << 34)])
def test_layers_whose_length_passes_64_bits(pkm, kw):
    """Rows brought by loads count 16-byte units in 32 bits; the product must not wrap to fewer."""
    assert attend(pkm, paged(pkm, **{"page_size": 12, **kw})) == UNSUPPORTED
    assert attend(pkm, quant(pkm, **kw)) == UNSUPPORTED


def test_longest_layer_for_loads(pkm):
    units = 2 ** 32 - 2
    for make, unit, slot in ((paged, 8, 576), (quant, 16, 656)):
        for over, status in ((0, UNSUPPORTED), (1, GOES_ON)):
            cache = make(pkm, page_size=12, num_pages=1,
                         page_stride=units * unit - 12 * slot - over * unit)
            assert attend(pkm, cache) == status
