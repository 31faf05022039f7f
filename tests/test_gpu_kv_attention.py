"""GPU: attention of new tokens over the paged K/V cache, with and without a window, against the
definition in 64 bits (tolerances: KvProblem.reference)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from kv_util import LSE_FILL, OUT_FILL, DeviceKv, assert_kv_close, check, make_kv
from spec_util import NAN_BF16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_mla_gb300  # noqa: F401


@pytest.mark.parametrize("size", [64, 128])
@pytest.mark.parametrize("ctx", [0, 1, 127, 128, 129, 700])
def test_one_token(ctx, size):
    check(make_kv(ctx, [ctx], [1], 8, 2, size, 16))


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 4), (8, 1), (6, 2), (20, 4), (71, 1), (128, 1),
                                            (96, 1), (130, 2), (64, 8)])
def test_groups_of_heads(heads, kv_heads):
    check(make_kv(heads, [200, 3, 77], [1, 5, 40], heads, kv_heads, 128, 32))


@pytest.mark.parametrize("page", [1, 4, 8, 12, 16, 24, 40, 64, 96, 128, 192, 256, 300])
def test_pages(page):
    check(make_kv(page, [0, 61, 333], [150, 7, 1], 8, 2, 128, page))


@pytest.mark.parametrize("size", [64, 128])
@pytest.mark.parametrize("layout", ["page", "plane", "slot"])
def test_layouts_and_padding(layout, size):
    check(make_kv(5, [90, 17], [33, 1], 12, 3, size, 16, layout=layout, pad=8), fused=True)


@pytest.mark.parametrize("new", [[1, 2, 3, 0, 0, 31], [32, 33, 63, 64, 65], [127, 128, 129], [255, 256, 257],
                                 [1000], [0, 0, 513, 0]])
@pytest.mark.parametrize("heads,kv_heads,size", [(8, 2, 128), (5, 1, 64)])
def test_chunks(new, heads, kv_heads, size):
    gen = np.random.default_rng(sum(new))
    check(make_kv(sum(new), gen.integers(0, 300, len(new)).tolist(), new, heads, kv_heads, size, 32))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 0), (128, 4), (129, 130), (300, 1),
                                          (5000, 9), (2 ** 31 - 1, 2 ** 31 - 1), (100, 2000)])
@pytest.mark.parametrize("size", [64, 128])
def test_window(window, sinks, size):
    p = make_kv(window % 97 + sinks % 89, [0, 1, 700, 1500], [200, 1, 90, 1], 8, 2, size, 16, window, sinks)
    d = check(p)
    if window >= 1790:
        full = make_kv(window % 97 + sinks % 89, p.ctx, p.new, 8, 2, size, 16)
        f = check(full)
        assert torch.equal(f.out, d.out) and torch.equal(f.lse, d.lse)


@pytest.mark.parametrize("page", [8, 12, 128])
def test_window_reads_nothing_between(page):
    """Pages between the first tokens and the window were given back: their table entries name no
    page of the cache."""
    p = make_kv(3, [2000, 900], [40, 1], 8, 2, 128, page, window=130, sinks=5)
    for b, c in enumerate(p.ctx):
        first, last = -(-p.sinks // page), (c + 1 - p.window) // page
        for lp in range(first, last):
            p.cache[:, p.table[b, lp]] = NAN_BF16
            p.table[b, lp] = 0xFFFFFFF0
    check(p)


@pytest.mark.parametrize("seed,batch,ctx_hi,new_hi,heads,kv_heads,size,page", [
    (1, 40, 900, 1, 32, 8, 128, 64), (2, 9, 5000, 1, 8, 1, 128, 128), (3, 70, 300, 12, 10, 2, 64, 16),
    (4, 6, 1500, 300, 16, 4, 128, 128), (5, 3, 20000, 2, 4, 2, 64, 32), (6, 300, 60, 3, 4, 1, 64, 8)])
def test_ragged_batches(seed, batch, ctx_hi, new_hi, heads, kv_heads, size, page):
    gen = np.random.default_rng(seed)
    ctx = gen.integers(0, ctx_hi + 1, batch).tolist()
    new = gen.integers(0 if batch > 8 else 1, new_hi + 1, batch).tolist()
    check(make_kv(seed, ctx, new, heads, kv_heads, size, page))
    check(make_kv(seed, ctx, new, heads, kv_heads, size, page, window=100, sinks=3))


def test_large_scores_and_negative_scale():
    """Weights of one key alone, maxima that grow along the keys."""
    p = make_kv(8, [600], [20], 8, 2, 128, 16, q_std=30.0)
    check(p)
    check(make_kv(8, [600], [20], 8, 2, 128, 16, scale=-0.3))
    check(make_kv(8, [600], [20], 8, 2, 128, 16, scale=0.0))


@pytest.mark.parametrize("value", [0x7F80, 0xFF80, 0x7FC0, 0xFF7F, 0x7F7F])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 2)])
def test_values_that_are_not_attended(value, window, sinks):
    """Infinities, NaN and the type's largest values in keys and values of later tokens, and of
    those between the first tokens and the window."""
    p = make_kv(9, [140], [90], 8, 2, 128, 16, window, sinks)
    clean = make_kv(9, [140], [90], 8, 2, 128, 16, window, sinks)
    at = [215, 216, 229] if window == 0 else [5, 60, 229]
    for t in at:
        p.cache[p.layer, p.table[0, t // 16], :, t % 16, 3:200:5] = value
    touched = p.seen(0)[:, at].any(1)
    assert touched.any() and not touched.all()
    d = DeviceKv(p)
    d.run()
    out, lse, status = d.results()
    assert status == 0
    assert_kv_close(clean, out, lse, rows=np.flatnonzero(~touched))


@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 4)])
def test_values_that_are_attended(window, sinks):
    """An infinity or NaN among the values of a token: in that column of the rows that attend it
    (their keys are finite), and nowhere else."""
    p = make_kv(10, [130], [150], 4, 2, 128, 16, window, sinks)
    row = {3: (0, 0x7F80), 100: (7, 0xFF80), 200: (130, 0x7FC0), 201: (130, 0x7F80), 231: (77, 0x7F80),
           240: (77, 0xFF80)}
    for t, (c, v) in row.items():
        p.cache[p.layer, p.table[0, t // 16], 1, t % 16, c] = v
    check(p)


def test_page_out_of_range():
    """Reported, and the other requests' rows are right."""
    for page in (12, 16):
        p = make_kv(11, [300, 100, 40], [2, 30, 1], 8, 2, 128, page)
        good = p.reference()
        p.table[1, 3] = 0x7FFFFFFF
        d = DeviceKv(p)
        d.run()
        out, lse, status = d.results()
        assert status == 4
        assert_kv_close(p, out, lse, good, rows=np.r_[0:2, 32:33])


def test_table_too_short():
    import paged_kv_mla_gb300 as pkm
    from gpu_util import dev
    p = make_kv(12, [300, 100], [2, 1], 8, 2, 128, 16)
    good = p.reference()
    d = DeviceKv(p)
    d.desc.page_table = dev(p.table[:, :18])  # the first request's last page is missing
    pkm.kv_attention_paged(d.q, d.offsets, p.scale, d.desc, p.layer, d.out, d.workspace, d.lse, d.status)
    out, lse, status = d.results()
    assert status == 4
    assert_kv_close(p, out, lse, good, rows=[2])


def test_rows_outside_the_requests():
    """Offsets that begin behind row 0 and end before the last."""
    import paged_kv_mla_gb300 as pkm
    from gpu_util import dev
    p = make_kv(13, [50, 300], [70, 3], 8, 2, 128, 16)
    d = DeviceKv(p)
    q = torch.cat([d.q[:5], d.q, d.q[:9]])
    out = torch.full((p.rows + 14, 8, 128), OUT_FILL, dtype=torch.int16, device="cuda")
    lse = torch.full((p.rows + 14, 8), LSE_FILL, dtype=torch.float32, device="cuda")
    ws = torch.empty(pkm.kv_attention_paged_workspace_size(p.rows + 14, 8, 2, 128), dtype=torch.uint8, device="cuda")
    pkm.kv_attention_paged(q, dev(p.offsets + np.uint32(5)), p.scale, d.desc, p.layer, out, ws, lse, d.status)
    o, l = out.cpu().numpy().view(np.uint16), lse.cpu().numpy()
    assert d.status.item() == 0
    assert (np.delete(o, np.s_[5:5 + p.rows], 0) == OUT_FILL).all()
    assert (np.delete(l, np.s_[5:5 + p.rows], 0) == LSE_FILL).all()
    assert_kv_close(p, o[5:], l[5:])
    # offsets that go past the last row
    short = DeviceKv(p)
    pkm.kv_attention_paged(short.q[:60], short.offsets, p.scale, short.desc, p.layer, short.out[:60],
                           short.workspace, short.lse[:60], short.status)
    o, l, status = short.results()
    assert status == 0 and (o[60:] == OUT_FILL).all()
    # positions of rows and lengths of requests as before: the first 60 rows of the first request
    assert_kv_close(p, o, l, rows=np.arange(60))


def test_same_bits_twice_and_without_lse():
    p = make_kv(14, [3000, 10, 900], [1, 200, 33], 16, 4, 128, 64)
    d = check(p)
    first, lse = d.out.clone(), d.lse.clone()
    d.out.fill_(1)
    d.run(workspace=d.new_workspace(), lse=False)
    torch.cuda.synchronize()
    assert torch.equal(d.out, first) and torch.equal(d.lse, lse)


def test_another_stream_and_a_graph():
    p = make_kv(15, [1000, 20], [3, 120], 8, 2, 128, 64)
    d = DeviceKv(p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        d.run()
    s.synchronize()
    out, lse, status = d.results()
    assert status == 0
    assert_kv_close(p, out, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.run()
    p2 = make_kv(16, [900, 50], [3, 120], 8, 2, 128, 64)  # the same pages at least
    other = DeviceKv(p2)
    assert other.cache.shape[1] <= d.cache.shape[1] and other.table.shape[1] <= d.table.shape[1]
    d.cache[:, :other.cache.shape[1]].copy_(other.cache)
    d.table[:, :other.table.shape[1]].copy_(other.table)
    d.q.copy_(other.q)
    d.lengths.copy_(other.lengths)
    graph.replay()
    out, lse, status = d.results()
    assert status == 0
    assert_kv_close(p2, out, lse)


def test_two_calls_at_once():
    """Two streams, a workspace each."""
    ps = [make_kv(20 + i, [2000, 100], [1, 150], 8, 2, 128, 64) for i in range(2)]
    ds = [DeviceKv(p) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(5):
        for d, s in zip(ds, streams):
            d.run(stream=s)
    for p, d in zip(ps, ds):
        out, lse, status = d.results()
        assert status == 0
        assert_kv_close(p, out, lse)


def test_positions_past_31_bits():
    """A history of four thousand million tokens, most of them given back: the window's pages alone
    are there."""
    import paged_kv_mla_gb300 as pkm
    size, page, width = 64, 1 << 14, 1 << 18
    c, n = 4294967000, 9
    p = make_kv(17, [296], [n], 4, 2, size, 1024, window=200, sinks=3)  # the same keys, at small positions
    d = DeviceKv(p)
    rows = d.cache[p.layer, int(p.table[0, 0].view(np.int32))]  # [planes, slots, row]
    table = torch.full((1, width), -16, dtype=torch.int32, device="cuda")
    cache = torch.full((1, 3, 2, page, 2 * size), -1, dtype=torch.int16, device="cuda")
    first = c - 296
    for t in list(range(3)) + list(range(first + 90, c + n)):
        table[0, t // page] = t // page % 2 if t > 10 else 2
    src = rows[:, :296 + n, :]
    cache[0, 2, :, :3] = src[:, :3]
    for j in range(90, 296 + n):
        t = first + j
        cache[0, t // page % 2, :, t % page] = src[:, j]
    desc = pkm.PagedCache(data=cache, page_table=table, layer_stride=0, page_stride=cache.stride(1),
                          kv_stride=cache.stride(2), slot_stride=cache.stride(3), num_layers=1, num_pages=3,
                          page_size=page, row_elems=2 * size,
                          cache_lengths=torch.tensor([c - 2 ** 32], dtype=torch.int32, device="cuda"))
    pkm.kv_window_attention_paged(d.q, d.offsets, p.scale, 200, 3, desc, 0, d.out, d.workspace, d.lse, d.status)
    out, lse, status = d.results()
    assert status == 0
    assert_kv_close(p, out, lse)
