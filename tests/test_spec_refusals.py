"""Refusals of the speculative-decoding entry points: a status before any CUDA call, so they
run without a GPU."""
from __future__ import annotations

import pytest
import torch

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def pkm():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_mla_gb300
    return paged_kv_mla_gb300


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def b16(*shape):
    return torch.zeros(shape, dtype=torch.int16)




def paged(pkm, cols=576, **kw):
    base = dict(data=b16(4 * 16 * cols), page_table=i32(2, 4), layer_stride=4 * 16 * cols,
                page_stride=16 * cols, slot_stride=cols, num_layers=1, num_pages=4, page_size=16,
                row_elems=cols, cache_lengths=i32(2))
    base.update(kw)
    return pkm.PagedCache(**base)


def quant(pkm, rank=512, rope=64, **kw):
    slot = (rank + 2 * rope + rank // 32 + 15) // 16 * 16
    base = dict(data=torch.zeros(4 * 16 * slot, dtype=torch.uint8), page_table=i32(2, 4),
                layer_stride=4 * 16 * slot, page_stride=16 * slot, slot_stride=slot, num_layers=1,
                num_pages=4, page_size=16, kv_lora_rank=rank, rope_dim=rope, cache_lengths=i32(2))
    base.update(kw)
    return pkm.QuantCache(**base)


def attention(pkm, cache, rank=512, rope=64, rows=3, heads=2, q=None, out=None, ws=None,
              scale=1.0, mask=None, layer=0, offsets=None):
    q = b16(rows, heads, rank + rope) if q is None else q
    out = b16(rows, heads, rank) if out is None else out
    if ws is None:
        n = pkm.mla_tree_attention_paged_workspace_size(rows, heads, rank)
        raw = torch.zeros(n + 256, dtype=torch.uint8)
        ws = raw[-raw.data_ptr() % 256:][:n]
    offsets = i32(3) if offsets is None else offsets
    if isinstance(cache, pkm.QuantCache):
        return pkm.mla_tree_attention_paged_qcache(q, offsets, scale, cache, layer, out, ws,
                                                   tree_mask=mask, stream=0, check=False)
    return pkm.mla_tree_attention_paged(q, offsets, scale, cache, layer, rank, rope, out, ws,
                                        tree_mask=mask, stream=0, check=False)


@pytest.mark.parametrize("kw,status", [
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(layer=1), INVALID), (dict(rank=448, rope=64), INVALID),  # row_elems differs
    (dict(ws=torch.zeros(256, dtype=torch.uint8)), INVALID),
    (dict(mask=torch.zeros(3, 0, dtype=torch.int32)), INVALID),  # not "no mask"
    (dict(mask=torch.zeros(2, 1, dtype=torch.int32)), INVALID),
    (dict(out=torch.zeros(2, 2, 512, dtype=torch.int16)), INVALID),
])
def test_attention_arguments(pkm, kw, status):
    assert attention(pkm, paged(pkm), **kw) == status


@pytest.mark.parametrize("field,value", [
    ("num_pages", 0), ("page_size", 0), ("page_size", -8), ("num_layers", 0), ("slot_stride", 577),
    ("page_stride", 12), ("layer_stride", -8), ("cache_lengths", None)])
def test_attention_cache(pkm, field, value):
    assert attention(pkm, paged(pkm, **{field: value})) == INVALID
    if field != "slot_stride":
        assert attention(pkm, quant(pkm, **{field: value if value != 577 else 600})) == INVALID


@pytest.mark.parametrize("rank,rope", [(32, 64), (576, 0), (520, 56), (512, 72), (64, 520)])
def test_attention_sizes(pkm, rank, rope):
    assert attention(pkm, paged(pkm, rank + rope), rank, rope) == UNSUPPORTED


@pytest.mark.parametrize("rank,rope", [(64, 64), (640, 64), (512, 72), (128, 12)])
def test_attention_quantised_sizes(pkm, rank, rope):
    assert attention(pkm, quant(pkm, rank, rope), rank, rope) == UNSUPPORTED


def test_attention_alignment_and_null(pkm):
    big = b16(3 * 2 * 576 + 8).view(torch.uint8)
    c = paged(pkm)
    import ctypes
    for q, out in ((big[2:], None), (None, big[8:])):
        cs = c.c_struct()
        ws = torch.zeros(pkm.mla_tree_attention_paged_workspace_size(3, 2, 512) + 256, dtype=torch.uint8)
        ws = ws[-ws.data_ptr() % 256:]
        code = pkm._lib.mla_tree_attention_paged(
            (q if q is not None else big).data_ptr(), i32(3).data_ptr(), 2, 3, 2, 512, 64, 1.0, None, 0,
            ctypes.byref(cs), 0, (out if out is not None else big).data_ptr(), None, ws.data_ptr(),
            ws.numel(), None, None)
        assert code == INVALID
    cs = c.c_struct()
    args = [big.data_ptr(), i32(3).data_ptr(), 2, 3, 2, 512, 64, 1.0, None, 0, ctypes.byref(cs), 0,
            big.data_ptr(), None, ws.data_ptr(), ws.numel(), None, None]
    for null in (0, 1, 10, 12, 14):
        bad = list(args)
        bad[null] = None
        assert pkm._lib.mla_tree_attention_paged(*bad) == INVALID
    bad = list(args)
    bad[14] += 16  # workspace not 256-byte aligned
    assert pkm._lib.mla_tree_attention_paged(*bad) == INVALID
    bad = list(args)
    bad[3] = bad[4] = 1 << 16  # more than 2^31 query rows
    assert pkm._lib.mla_tree_attention_paged(*bad) == UNSUPPORTED
    for at, value in ((2, -1), (3, -1), (4, 0), (5, 0), (6, -8)):
        bad = list(args)
        bad[at] = value
        assert pkm._lib.mla_tree_attention_paged(*bad) == INVALID


def test_nothing_to_do_is_fine(pkm):
    empty = b16(0, 2, 576)
    assert attention(pkm, paged(pkm), rows=0, q=empty, out=b16(0, 2, 512),
                     ws=torch.zeros(0, dtype=torch.uint8)) == 0
    assert attention(pkm, paged(pkm), offsets=i32(1)) == 0
    f = torch.zeros(4, 16)
    assert pkm.mla_rope_heads(b16(0, 2, 16), i32(0), f, b16(0, 2, 16), stream=0) == 0
    assert pkm.mla_cache_compact_paged(paged(pkm), 0, 0, i32(2, 3), i32(2), stream=0) == 0


def test_workspace_size(pkm):
    f = pkm.mla_tree_attention_paged_workspace_size
    assert f(-1, 1, 64) == 0 and f(1, 0, 64) == 0 and f(1, 1, 0) == 0
    assert f(1, 16, 512) < f(8, 16, 512) == f(4096, 128, 512)


def rope(pkm, x, y, positions=None, freqs=None, half=False):
    rows, P = x.shape[0], x.shape[-1]
    return pkm.mla_rope_heads(x, i32(rows) if positions is None else positions,
                              torch.zeros(4, P) if freqs is None else freqs, y, half=half,
                              stream=0, check=False)


def test_rope_arguments(pkm):
    x = b16(3, 4, 16)
    assert rope(pkm, x, b16(3, 4, 24)) == INVALID            # shapes differ
    assert rope(pkm, x, b16(3, 4, 16), positions=i32(2)) == INVALID
    assert rope(pkm, x, b16(3, 4, 16), freqs=torch.zeros(4, 8)) == INVALID
    assert rope(pkm, b16(3, 4, 32)[..., ::2], b16(3, 4, 16)) == INVALID   # columns apart
    assert rope(pkm, b16(3, 4, 20)[..., :16], b16(3, 4, 16)) == INVALID   # stride 20
    assert rope(pkm, b16(3, 4, 32)[..., 4:20], b16(3, 4, 16)) == INVALID  # 8-byte aligned
    assert rope(pkm, x, b16(3, 1, 16).expand(3, 4, 16)) == INVALID        # heads overlap
    assert rope(pkm, x, b16(1, 4, 16).expand(3, 4, 16)) == INVALID        # rows overlap
    t = b16(3, 4, 64)
    assert rope(pkm, t[..., :16], torch.as_strided(t, (3, 4, 16), (64, 192, 1))) == INVALID
    assert rope(pkm, b16(2, 2, 12), b16(2, 2, 12)) == INVALID             # strides of 12
    assert rope(pkm, b16(2, 2, 16)[..., :12], b16(2, 2, 16)[..., :12]) == UNSUPPORTED
    assert rope(pkm, b16(2, 2, 264), b16(2, 2, 264)) == UNSUPPORTED


def test_compact_arguments(pkm):
    acc, cnt, new = i32(2, 3), i32(2), i32(2)

    def call(cache, begin=0, count=1, acc=acc, cnt=cnt, new=new):
        f = pkm.mla_cache_compact_paged_qcache if isinstance(cache, pkm.QuantCache) \
            else pkm.mla_cache_compact_paged
        return f(cache, begin, count, acc, cnt, new, stream=0, check=False)

    for make in (paged, quant):
        c = make(pkm)
        assert call(c, begin=1) == INVALID and call(c, count=2) == INVALID
        assert call(c, count=-1) == INVALID and call(c, acc=i32(2, 0)) == INVALID
        assert call(c, new=c.cache_lengths) == INVALID
        assert call(make(pkm, cache_lengths=None)) == INVALID
        assert call(make(pkm, page_size=0)) == INVALID
        assert call(make(pkm, slot_stride=8 + 4)) == INVALID
    assert call(paged(pkm, row_elems=20)) == UNSUPPORTED
    assert call(quant(pkm, 64)) == UNSUPPORTED


def test_cache_write_at_needs_positions(pkm):
    c = paged(pkm)
    lat, g, f = b16(3, 576), torch.zeros(512), torch.zeros(8, 64)
    assert pkm.mla_cache_write_paged_at(lat, i32(3), None, g, 1e-6, f, c, 0, 512, 64, stream=0,
                                        check=False) == INVALID
    assert pkm.mla_cache_write_paged_qcache_at(lat, i32(3), None, g, 1e-6, f, quant(pkm), 0, stream=0,
                                               check=False) == INVALID
    assert pkm.mla_cache_write_paged_at(lat, i32(3), i32(3), g, 1e-6, f, paged(pkm, row_elems=80), 0,
                                        512, 64, stream=0, check=False) == INVALID


def test_views_that_the_calls_cannot_see(pkm):
    """Strided tensors and other element sizes, which the C call would read as plain arrays."""
    q = b16(3, 2, 640)[:, :, :576]
    assert attention(pkm, paged(pkm), q=q) == INVALID
    assert attention(pkm, paged(pkm), out=b16(3, 2, 576)[:, :, :512]) == INVALID
    assert attention(pkm, paged(pkm), mask=torch.zeros(3, 1, dtype=torch.int64)) == INVALID
    assert attention(pkm, quant(pkm), q=q) == INVALID
    cache = paged(pkm)
    for accepted, counts in ((i32(2, 8)[:, :3], i32(2)), (i32(3, 4), i32(3)), (i32(2, 4), i32(1)),
                             (i32(2, 4).long(), i32(2))):
        assert pkm.mla_cache_compact_paged(cache, 0, 1, accepted, counts, stream=0,
                                           check=False) == INVALID
    x = b16(3, 2, 64)
    for positions in (i32(6)[::2], i32(3).long()):
        assert pkm.mla_rope_heads(x, positions, torch.zeros(8, 64), x, stream=0,
                                  check=False) == INVALID
        assert pkm.mla_cache_write_paged_at(b16(3, 576), i32(3), positions, torch.ones(512), 1e-6,
                                            torch.zeros(8, 64), cache, 0, 512, 64, stream=0,
                                            check=False) == INVALID


def test_layers_too_long_for_loads(pkm):
    """Rows brought by loads count 16-byte units in 32 bits."""
    far = dict(page_stride=1 << 35, layer_stride=1 << 37)
    assert attention(pkm, paged(pkm, page_size=12, **far)) == UNSUPPORTED
    assert attention(pkm, quant(pkm, **far)) == UNSUPPORTED
