"""Refusals of the entry points on the paged K/V cache: a status before any CUDA call, so they run
without a GPU."""
from __future__ import annotations

import ctypes

import pytest
import torch

from test_spec_refusals import INVALID, UNSUPPORTED, b16, i32

GOES_ON = 3  # PKM_ERR_CUDA: nothing was found, and nothing may be launched


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_mla_gb300
    return paged_kv_mla_gb300


@pytest.fixture()
def pkm(lib, monkeypatch):
    """The binding with its checks alone, on host memory taken for the device's."""
    monkeypatch.setattr(lib, "_here", lambda device: True)
    lib._lib.pkm_checks_only(1)
    yield lib
    lib._lib.pkm_checks_only(0)


def cache(pkm, row=512, **kw):
    base = dict(data=b16(4 * 2 * 16 * row), page_table=i32(2, 4), layer_stride=4 * 2 * 16 * row,
                page_stride=2 * 16 * row, kv_stride=16 * row, slot_stride=row, num_layers=1, num_pages=4,
                page_size=16, row_elems=row, cache_lengths=i32(2))
    base.update(kw)
    return pkm.PagedCache(**base)


def attention(pkm, c, rows=3, heads=8, size=128, q=None, out=None, ws=None, lse=None, scale=1.0, layer=0,
              offsets=None, window=None, sinks=0):
    q = b16(rows, heads, size) if q is None else q
    out = b16(rows, heads, size) if out is None else out
    if ws is None:
        n = pkm.kv_attention_paged_workspace_size(rows, heads, max(c.row_elems // size, 1), size)
        n = n or 4096  # nothing is said of heads that are refused
        raw = torch.zeros(n + 256, dtype=torch.uint8)
        ws = raw[-raw.data_ptr() % 256:][:n]
    offsets = i32(3) if offsets is None else offsets
    if window is not None:
        return pkm.kv_window_attention_paged(q, offsets, scale, window, sinks, c, layer, out, ws, lse=lse,
                                             stream=0, check=False)
    return pkm.kv_attention_paged(q, offsets, scale, c, layer, out, ws, lse=lse, stream=0, check=False)


@pytest.mark.parametrize("kw,status", [
    (dict(), GOES_ON), (dict(window=1), GOES_ON), (dict(window=7, sinks=3), GOES_ON),
    (dict(window=0), INVALID), (dict(window=-1), INVALID), (dict(window=5, sinks=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("-inf")), INVALID), (dict(scale=-1.0), GOES_ON),
    (dict(layer=1), INVALID), (dict(ws=torch.zeros(256, dtype=torch.uint8)), INVALID),
    (dict(heads=6), INVALID),                       # not a multiple of the four heads of keys
    (dict(heads=4), GOES_ON), (dict(heads=512), GOES_ON), (dict(heads=516), UNSUPPORTED),
    (dict(out=b16(2, 8, 128)), INVALID), (dict(out=b16(3, 8, 256)[..., :128]), INVALID),
    (dict(lse=torch.zeros(3, 4)), INVALID), (dict(lse=torch.zeros(3, 8, dtype=torch.float64)), INVALID),
    (dict(q=torch.zeros(3, 8, 128)), INVALID), (dict(q=b16(24, 128)), INVALID),
    (dict(q=b16(3, 8, 136)[..., :128]), GOES_ON), (dict(q=b16(3, 8, 132)[..., :128]), INVALID),
    (dict(q=b16(3, 8, 256)[..., ::2]), INVALID), (dict(q=b16(3, 1, 128).expand(3, 8, 128)), INVALID),
    (dict(q=b16(8, 3, 128).transpose(0, 1)), GOES_ON), (dict(q=b16(3, 8, 144)[..., 4:132]), INVALID),
    (dict(offsets=i32(4)), INVALID),                # more requests than table rows
    (dict(offsets=i32(3).long()), INVALID),
])
def test_attention_arguments(pkm, kw, status):
    assert attention(pkm, cache(pkm), **kw) == status


@pytest.mark.parametrize("field,value", [
    ("num_pages", 0), ("page_size", 0), ("page_size", -8), ("num_layers", 0), ("slot_stride", 516),
    ("page_stride", 12), ("layer_stride", -8), ("cache_lengths", None), ("kv_stride", 0), ("kv_stride", 504),
    ("cache_lengths", i32(1)), ("page_table", i32(1, 4)), ("page_table", i32(2, 0)), ("row_elems", 500)])
def test_the_cache(pkm, field, value):
    c = cache(pkm, **{field: value})
    assert attention(pkm, c) == INVALID and attention(pkm, c, window=9) == INVALID
    assert rope(pkm, c) == INVALID


@pytest.mark.parametrize("size,status", [(32, UNSUPPORTED), (64, GOES_ON), (128, GOES_ON), (256, UNSUPPORTED)])
def test_attention_sizes(pkm, size, status):
    assert attention(pkm, cache(pkm, 2 * size), size=size) == status


def test_pages_of_any_size_go_on(pkm):
    for page in (1, 7, 12, 16, 100, 128, 300):
        assert attention(pkm, cache(pkm, page_size=page)) == GOES_ON
    assert attention(pkm, cache(pkm, page_stride=1 << 40)) == GOES_ON  # past a tensor map: row by row
    q = torch.as_strided(b16(128), (1, 8, 128), (8, 0, 1))
    assert attention(pkm, cache(pkm), rows=1, q=q) == INVALID  # one head's elements for all


def test_attention_null_alignment_and_limits(pkm):
    import paged_kv_mla_gb300 as m
    c = cache(pkm)
    cs = c.c_struct()
    q, out = b16(3 * 8 * 128 + 64), b16(3 * 8 * 128 + 64)
    ws = torch.zeros(m.kv_attention_paged_workspace_size(3, 8, 4, 128) + 256, dtype=torch.uint8)
    ws = ws[-ws.data_ptr() % 256:]
    args = [q.data_ptr(), 1024, 128, i32(3).data_ptr(), 2, 3, 8, 4, 128, 1.0, ctypes.byref(cs), 0, out.data_ptr(),
            None, ws.data_ptr(), ws.numel(), None, None]
    f = m._lib.kv_attention_paged

    def call(**kw):
        a = list(args)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    assert call() == GOES_ON
    for at in (0, 3, 10, 12, 14):
        assert call(**{f"_{at}": None}) == INVALID
    assert call(_0=q.data_ptr() + 8) == INVALID and call(_12=out.data_ptr() + 8) == INVALID
    assert call(_14=ws.data_ptr() + 16) == INVALID
    assert call(_1=1023) == INVALID and call(_2=-128) == INVALID and call(_1=8) == INVALID
    for at, value in ((4, -1), (5, -1), (6, 0), (7, 0), (8, 0), (6, -8)):
        assert call(**{f"_{at}": value}) == INVALID
    assert call(_5=1 << 28, _1=1 << 20) == UNSUPPORTED      # 2^31 query rows
    assert call(_1=1 << 39) == UNSUPPORTED                  # a stride past a tensor map
    assert call(_4=0) == 0 and call(_5=0) == 0              # nothing to do
    assert call(_4=0, _0=None, _10=None) == 0


def test_workspace_size(lib):
    f = lib.kv_attention_paged_workspace_size
    assert f(-1, 8, 2, 128) == 0 and f(1, 0, 1, 128) == 0 and f(1, 8, 0, 128) == 0 and f(1, 8, 2, 0) == 0
    assert f(1, 7, 2, 128) == 0 and f(1, 129, 1, 64) == 0
    assert 0 < f(1, 8, 2, 128) < f(16, 8, 2, 128) < f(33, 8, 2, 128) == f(100000, 8, 2, 128)


def rope(pkm, c, rows=3, heads=8, kv=4, size=128, P=None, axes=1, half=False, **kw):
    P = size if P is None else P
    a = dict(q=b16(rows, heads, size), q_out=b16(rows, heads, size), k=b16(rows, kv, size), v=b16(rows, kv, size),
             positions=i32(axes, rows), freqs=torch.zeros(16, P), offsets=i32(3), pair_axes=None)
    a.update(kw)
    return pkm.kv_rope_paged(a["offsets"], a["positions"], a["freqs"], c, kw.get("layer", 0), kv, q=a["q"],
                             q_out=a["q_out"], k=a["k"], v=a["v"], pair_axes=a["pair_axes"], half=half, stream=0,
                             check=False)


@pytest.mark.parametrize("kw,status", [
    (dict(), GOES_ON), (dict(q=None, q_out=None), GOES_ON), (dict(k=None), GOES_ON), (dict(k=None, v=None), GOES_ON),
    (dict(v=None), GOES_ON), (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(layer=1), INVALID),
    (dict(positions=i32(3)), GOES_ON), (dict(positions=i32(4)), INVALID), (dict(positions=i32(1, 1, 3)), INVALID),
    (dict(positions=i32(1, 3).long()), INVALID), (dict(positions=i32(2, 6)[:, ::2]), INVALID),
    (dict(axes=4), GOES_ON), (dict(axes=5), UNSUPPORTED), (dict(axes=0), INVALID),
    (dict(axes=3, pair_axes=[j % 3 for j in range(64)]), GOES_ON), (dict(axes=3, pair_axes=[0] * 63), INVALID),
    (dict(axes=3, pair_axes=[3] * 64), INVALID), (dict(axes=3, pair_axes=[-1] * 64), INVALID),
    (dict(axes=3, pair_axes=[300] * 64), INVALID), (dict(axes=3, pair_axes=["a"] * 64), INVALID),
    (dict(freqs=torch.zeros(16, 64)), GOES_ON), (dict(freqs=torch.zeros(16, 136)), INVALID),
    (dict(freqs=torch.zeros(16, 60)), UNSUPPORTED), (dict(freqs=torch.zeros(16)), INVALID),
    (dict(freqs=torch.zeros(0, 128)), INVALID), (dict(freqs=torch.zeros(16, 128, dtype=torch.float64)), INVALID),
    (dict(k=b16(3, 4, 64)), INVALID), (dict(k=b16(3, 5, 128)), INVALID), (dict(v=b16(2, 4, 128)), INVALID),
    (dict(k=torch.zeros(3, 4, 128)), INVALID), (dict(v=b16(3, 4, 256)[..., ::2]), INVALID),
    (dict(q=b16(3, 8, 64), q_out=b16(3, 8, 64)), INVALID), (dict(q_out=b16(3, 4, 128)), INVALID),
    (dict(q_out=b16(3, 1, 128).expand(3, 8, 128)), INVALID), (dict(q_out=b16(1, 8, 128).expand(3, 8, 128)), INVALID),
    (dict(k=b16(3, 1, 128).expand(3, 4, 128)), GOES_ON), (dict(q=b16(3, 8, 132)[..., :128]), INVALID),
    (dict(offsets=i32(4)), INVALID), (dict(kv=0, k=b16(3, 0, 128), v=b16(3, 0, 128)), INVALID),
])
def test_rope_arguments(pkm, kw, status):
    assert rope(pkm, cache(pkm), **kw) == status


def test_rope_sizes_and_planes(pkm):
    for size, status in ((8, GOES_ON), (104, GOES_ON), (256, GOES_ON), (264, UNSUPPORTED), (12, INVALID)):
        c = cache(pkm, 4 * size, page_stride=1 << 20, kv_stride=1 << 16, slot_stride=2048)
        assert rope(pkm, c, size=size, P=size // 8 * 8) == status
    assert rope(pkm, cache(pkm, slot_stride=504)) == INVALID           # slots overlap
    assert rope(pkm, cache(pkm, slot_stride=504, page_size=1)) == GOES_ON
    assert rope(pkm, cache(pkm, kv_stride=512)) == INVALID             # values of a slot are keys of the next
    assert rope(pkm, cache(pkm, kv_stride=512), v=None) == GOES_ON
    assert rope(pkm, cache(pkm, kv_stride=512, slot_stride=1024)) == GOES_ON
    # in place, with the same strides
    q = b16(3, 8, 128)
    assert rope(pkm, cache(pkm), q=q, q_out=q) == GOES_ON
    t = b16(3 * 8 * 256)
    a, b = torch.as_strided(t, (3, 8, 128), (1024, 128, 1)), torch.as_strided(t, (3, 8, 128), (2048, 256, 1))
    assert rope(pkm, cache(pkm), q=a, q_out=b) == INVALID


def test_rope_heads_of_a_row_are_counted(pkm):
    import paged_kv_mla_gb300 as m
    cs = cache(pkm).c_struct()
    t = b16(3 * 8 * 128)
    f = torch.zeros(16, 128)
    rest = [t.data_ptr(), 512, 128, t.data_ptr(), 512, 128, 4, 128, 128, i32(3).data_ptr(), 2, 1, i32(3).data_ptr(), 1,
            None, f.data_ptr(), 16, 0, ctypes.byref(cs), 0, None, None]
    for heads, status in ((2 ** 31 - 513 - 8, GOES_ON), (2 ** 31 - 512 - 8, UNSUPPORTED), (2 ** 31 - 1, UNSUPPORTED)):
        assert m._lib.kv_rope_paged(t.data_ptr(), heads * 128, 128, heads, t.data_ptr(), heads * 128, 128, *rest) == status


def test_nothing_to_do(lib):
    """No rows, or no requests: fine, and nothing is launched (nor is there a GPU)."""
    c = cache(lib)
    assert attention(lib, c, rows=0, ws=torch.zeros(0, dtype=torch.uint8)) == 0
    assert attention(lib, c, offsets=i32(1)) == 0
    assert rope(lib, c, rows=0) == 0 and rope(lib, c, offsets=i32(1)) == 0


@pytest.mark.parametrize("call", [attention, rope])
def test_host_memory_is_refused(lib, call):
    assert call(lib, cache(lib)) == INVALID
