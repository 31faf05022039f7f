"""GPU: the operators on the paged K/V cache far from ordinary sizes -- many items a block, offsets
and positions past 31 bits, values that are not finite in shared items, other orders of the queries,
workspaces and pages that calls and requests share."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from kv_util import LSE_FILL, OUT_FILL, DeviceKv, assert_kv_close, check, make_kv
from spec_util import bf16_value, freqs_table
from test_gpu_kv_rope import assert_turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_mla_gb300  # noqa: F401


@pytest.mark.parametrize("size,page,window,sinks", [(64, 128, 1024, 4), (128, 128, 0, 0), (64, 24, 500, 140)])
def test_many_single_tokens(size, page, window, sinks):
    """Several items a block, none of them short."""
    gen = np.random.default_rng(size + page)
    ctx = gen.integers(1500, 3000, 40).tolist()
    check(make_kv(30, ctx, [1] * 40, 32, 8, size, page, window, sinks, layers=1, layer=0))


@pytest.mark.parametrize("size,window,sinks", [(64, 0, 0), (128, 0, 0), (128, 200, 3), (64, 128, 128)])
def test_many_items_of_a_chunk(size, window, sinks):
    check(make_kv(31, [333], [1100], 48, 6, size, 64, window, sinks, layers=1, layer=0))


@pytest.mark.parametrize("size,ctx,new", [(64, 4000, 1), (128, 4000, 1), (64, 3500, 40), (128, 3500, 40),
                                          (64, 500, 200), (128, 500, 200)])
def test_not_finite_in_shared_items(size, ctx, new):
    """Infinities and NaN among values that all, some and none of the tokens attend, where several
    blocks share an item and where two stages are joined."""
    p = make_kv(32, [ctx], [new], 4, 1, size, 16, layers=1, layer=0)
    last = ctx + new - 1
    for t, c, v in [(3, 0, 0x7F80), (129, 7, 0xFF80), (ctx - 1, 9, 0x7FC0), (ctx - 1, 33, 0x7F80),
                    (ctx, 33, 0x7F80), (last, 40, 0xFF80), (last - new // 2, 41, 0x7F80), (last, 42, 0x7FC0),
                    (ctx, 50, 0x7F80), (last, 50, 0xFF80)]:
        p.cache[0, p.table[0, t // 16], 1, t % 16, c] = v
    check(p)


@pytest.mark.parametrize("page", [16, 12])
def test_offsets_past_31_bits(page):
    """Pages 2^30 elements apart: those of a request lie past 2^31 elements."""
    import paged_kv_mla_gb300 as pkm
    p = make_kv(33, [30], [9], 8, 2, 128, page, layers=1, layer=0)
    d = DeviceKv(p)
    pages, stride = p.cache.shape[1], (1 << 30) + 64
    far = torch.empty((pages - 1) * stride + 2 * page * 256, dtype=torch.int16, device="cuda")
    view = torch.as_strided(far, (pages, 2, page, 256), (stride, page * 256, 256, 1))
    view.copy_(d.cache[0])
    desc = pkm.PagedCache(data=far, page_table=d.table, layer_stride=0, page_stride=stride, kv_stride=page * 256,
                          slot_stride=256, num_layers=1, num_pages=pages, page_size=page, row_elems=256,
                          cache_lengths=d.lengths)
    pkm.kv_attention_paged(d.q, d.offsets, p.scale, desc, 0, d.out, d.workspace, d.lse, d.status)
    out, lse, status = d.results()
    assert status == 0
    assert_kv_close(p, out, lse)
    # keys turn in place, and values are written, in the same places
    freqs = torch.from_numpy(freqs_table(50, 64)).cuda()
    at = torch.arange(9, dtype=torch.int32, device="cuda") * 5
    v = torch.randint(-30000, 30000, (9, 2, 128), dtype=torch.int16, device="cuda")
    before = view.clone()
    pkm.kv_rope_paged(d.offsets, at, freqs, desc, 0, 2, v=v, dev_status=d.status)
    assert d.status.item() == 0
    cs = freqs.cpu().numpy().astype(np.float64)[at.cpu().numpy()][:, None]
    for i in range(9):
        where = int(p.table[0, (30 + i) // page]), (30 + i) % page
        assert_turned(*[x[where[0], 0, where[1]].cpu().numpy().view(np.uint16).reshape(1, 2, 128)
                        for x in (view, before)], cs[i:i + 1], 64, False)
        assert torch.equal(view[where[0], 1, where[1]], v[i].view(-1))
        before[where[0], :, where[1]] = view[where[0], :, where[1]]
    assert torch.equal(view, before)


def test_rows_past_31_bits():
    """Queries and outputs of more than 2^31 elements: 140 000 requests of one token, whose one key
    has all the weight."""
    import paged_kv_mla_gb300 as pkm
    n, heads, size = 140_000, 128, 128
    q = torch.zeros(n, heads, size, dtype=torch.bfloat16, device="cuda")
    q[-3:] = 1.0
    cache = torch.randn(7, 2, 8, size, device="cuda").bfloat16()
    table = (torch.arange(n, device="cuda", dtype=torch.int32) % 7).view(n, 1)
    offsets = torch.arange(n + 1, device="cuda", dtype=torch.int32)
    desc = pkm.PagedCache(data=cache, page_table=table, layer_stride=0, page_stride=2 * 8 * size, kv_stride=8 * size,
                          slot_stride=size, num_layers=1, num_pages=7, page_size=8, row_elems=size,
                          cache_lengths=torch.zeros(n, dtype=torch.int32, device="cuda"))
    out = torch.full_like(q, 7.0)
    lse = torch.full((n, heads), LSE_FILL, device="cuda")
    ws = torch.empty(pkm.kv_attention_paged_workspace_size(n, heads, 1, size), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkm.kv_attention_paged(q, offsets, 0.125, desc, 0, out, ws, lse, status)
    assert status.item() == 0
    page = table[:, 0].long()
    expected = cache[page, 1, 0]
    for at in range(0, n, 20_000):
        assert (out[at:at + 20_000] == expected[at:at + 20_000, None]).all()
    sums = torch.where(torch.arange(n, device="cuda") >= n - 3, cache[page, 0, 0].double().sum(1) * 0.125, 0.0)
    assert ((lse - sums[:, None]).abs() <= 2.0 ** -17 * cache[page, 0, 0].double().abs().sum(1)[:, None]).all()
    # the same rows turned: factors (0, 1) take (x0, x1) to (-x1, x0)
    freqs = torch.tensor([[0.0, 1.0] * (size // 2)], device="cuda")
    q[-5:] = torch.randn(5, heads, size, device="cuda").bfloat16()
    whole = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    slots = torch.empty(n, 2, size, dtype=torch.int16, device="cuda")
    desc = pkm.PagedCache(data=slots, page_table=torch.zeros(1, 1, dtype=torch.int32, device="cuda"), layer_stride=0,
                          page_stride=0, kv_stride=size, slot_stride=2 * size, num_layers=1, num_pages=1, page_size=n,
                          row_elems=size, cache_lengths=torch.zeros(1, dtype=torch.int32, device="cuda"))
    k = torch.randn(n, 1, size, device="cuda").bfloat16()
    pkm.kv_rope_paged(whole, torch.zeros(n, dtype=torch.int32, device="cuda"), freqs, desc, 0, 1, q=q, q_out=out, k=k,
                      v=k, dev_status=status)
    assert status.item() == 0

    def turned(x):
        return torch.stack([-x[..., 1::2], x[..., 0::2]], -1).flatten(-2)

    for at in range(0, n, 20_000):
        assert (out[at:at + 20_000] == turned(q[at:at + 20_000])).all()
    assert (slots[:, 0].view(torch.bfloat16) == turned(k[:, 0])).all()
    assert torch.equal(slots[:, 1], k[:, 0].view(torch.int16))


def test_positions_past_31_bits_in_pages_of_any_size():
    """A history of four thousand million tokens in pages of 12 345; keys turned and values written
    there first."""
    import paged_kv_mla_gb300 as pkm
    size, page, c, n = 64, 12345, 4294967000, 9
    p = make_kv(34, [296], [n], 4, 2, size, 1024, window=200, sinks=3)  # the same keys, at small positions
    d = DeviceKv(p)
    rows = d.cache[p.layer, int(p.table[0, 0].view(np.int32))]
    width = (c + n) // page + 1
    table = torch.full((1, width), -16, dtype=torch.int32, device="cuda")
    cache = torch.full((3, 2, page, 2 * size), -1, dtype=torch.int16, device="cuda")
    first = c - 296
    for t in list(range(3)) + list(range(first + 90, c + n)):
        table[0, t // page] = t // page % 2 if t > 10 else 2
    cache[2, :, :3] = rows[:, :3]
    for j in range(90, 296):
        t = first + j
        cache[t // page % 2, :, t % page] = rows[:, j]
    desc = pkm.PagedCache(data=cache, page_table=table, layer_stride=0, page_stride=cache.stride(0),
                          kv_stride=cache.stride(1), slot_stride=cache.stride(2), num_layers=1, num_pages=3,
                          page_size=page, row_elems=2 * size,
                          cache_lengths=torch.tensor([c - 2 ** 32], dtype=torch.int32, device="cuda"))
    # a turn by nothing: the new tokens' keys and values as they are
    freqs = torch.tensor([[1.0, 0.0] * (size // 2)], device="cuda")
    new = rows[:, 296:296 + n].reshape(2, n, 2, size)
    pkm.kv_rope_paged(d.offsets, torch.zeros(n, dtype=torch.int32, device="cuda"), freqs, desc, 0, 2, k=new[0],
                      v=new[1], half=True, dev_status=d.status)
    pkm.kv_window_attention_paged(d.q, d.offsets, p.scale, 200, 3, desc, 0, d.out, d.workspace, d.lse, d.status)
    out, lse, status = d.results()
    assert status == 0
    assert_kv_close(p, out, lse)


def test_graphs_that_share_a_workspace():
    """Captured one after the other, replayed in turn on one stream; each has its own results."""
    ds = [DeviceKv(make_kv(35, [3000, 20], [1, 90], 8, 2, 128, 64)),
          DeviceKv(make_kv(36, [10, 2500, 700], [5, 1, 85], 8, 2, 128, 16, window=900, sinks=2))]
    assert ds[0].workspace.numel() == ds[1].workspace.numel()
    graphs = []
    for d in ds:
        d.run(workspace=ds[0].workspace)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            d.run(workspace=ds[0].workspace)
    for _ in range(3):
        for d in ds:
            d.out_all.fill_(OUT_FILL)
            d.lse_all.fill_(LSE_FILL)
        for _ in range(20):
            for g in graphs:
                g.replay()
        for d in ds:
            out, lse, status = d.results()
            assert status == 0
            assert_kv_close(d.p, out, lse)


def test_a_padded_batch():
    """Requests of no tokens, whatever their lengths and pages, before, between and behind others:
    nothing is read or reported for them."""
    p = make_kv(37, [40, 50, 70, 0], [0, 33, 0, 0], 8, 2, 64, 16)
    p.table[[0, 2, 3]] = 0xFFFFFFFF
    d = DeviceKv(p)
    d.lengths[torch.tensor([0, 2, 3])] = -1
    d.run()
    out, lse, status = d.results()
    assert status == 0
    assert_kv_close(p, out, lse)


def test_rows_of_no_request():
    """Offsets that cover no row at all: nothing is written or reported."""
    import paged_kv_mla_gb300 as pkm
    p = make_kv(41, [30, 9], [5, 2], 8, 2, 64, 16)
    d = DeviceKv(p)
    for at in (0, 7, 3):
        d.offsets.fill_(at)
        d.run()
        pkm.kv_rope_paged(d.offsets, torch.zeros(7, dtype=torch.int32, device="cuda"),
                          torch.zeros(1, 64, device="cuda"), d.desc, p.layer, 2, q=d.q, q_out=d.out, dev_status=d.status)
    out, lse, status = d.results()
    assert status == 0 and (out == OUT_FILL).all() and (lse == LSE_FILL).all()
    assert torch.equal(d.cache, DeviceKv(p).cache)


@pytest.mark.parametrize("page", [1, 5, 8])
def test_windows_over_small_pages(page):
    check(make_kv(42, [700, 0, 90], [40, 3, 1], 8, 2, 64, page, window=150, sinks=9))


@pytest.mark.parametrize("size", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (130, 0), (300, 200), (1, 129)])
def test_heads_of_their_own_keys(size, window, sinks):
    """128 tokens a tile of queries, 256 an item, whose diagonal and edge lie in three tiles each."""
    check(make_kv(43, [126, 300, 1000], [770, 257, 129], 3, 3, size, 32, window=window, sinks=sinks))


def test_a_million_tokens_each():
    """512 requests of 2^20 tokens on one page: 33 million tiles of keys, whose line is cut with 64-bit
    products.  The page's keys count 8192 times each, so the weights are the page's."""
    import paged_kv_mla_gb300 as pkm
    n, heads, size, page, times = 512, 8, 64, 128, 8192
    gen = torch.Generator(device="cuda").manual_seed(44)
    cache = torch.randn(1, 2, page, heads * size, device="cuda", generator=gen).bfloat16()
    q = torch.randn(n, heads, size, device="cuda", generator=gen).bfloat16()
    table = torch.zeros(n, times, dtype=torch.int32, device="cuda")
    offsets = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    desc = pkm.PagedCache(data=cache, page_table=table, layer_stride=0, page_stride=0, kv_stride=page * heads * size,
                          slot_stride=heads * size, num_layers=1, num_pages=1, page_size=page, row_elems=heads * size,
                          cache_lengths=torch.full((n,), page * times - 1, dtype=torch.int32, device="cuda"))
    out, lse = torch.zeros_like(q), torch.zeros(n, heads, device="cuda")
    ws = torch.empty(pkm.kv_attention_paged_workspace_size(n, heads, heads, size), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkm.kv_attention_paged(q, offsets, size ** -0.5, desc, 0, out, ws, lse, status)
    assert status.item() == 0
    k, v = cache[0].double().view(2, page, heads, size)
    s = torch.einsum("nhc,thc->nht", q.double(), k) * size ** -0.5
    e = size * 2.0 ** -24 * (torch.einsum("nhc,thc->nht", q.double().abs(), k.abs()) * size ** -0.5).amax(-1)
    w = s.softmax(-1)
    ref, spread = torch.einsum("nht,thc->nhc", w, v), torch.einsum("nht,thc->nhc", w, v.abs())
    # besides a short sum's errors: the running fp32 sum of a stage, which has every other tile, takes
    # 16 keys at a time, 2^15 times, each at most 2^-23 off if the MMAs cut off; the weights' sum
    # takes a tile at a time, rounded
    long = 2.0 ** -8
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12 + 2 * e[..., None] + 2 * long) * spread
    assert ((out.double() - ref).abs() <= tol).all()
    exact = torch.logsumexp(s, -1) + np.log(times)
    assert ((lse.double() - exact).abs() <= e + long + 2.0 ** -20 * (1 + exact.abs())).all()


@pytest.mark.parametrize("half", [False, True])
def test_inputs_that_heads_and_rows_share(half):
    """Queries, keys and values broadcast over heads or rows: as if they were written out."""
    import paged_kv_mla_gb300 as pkm
    rows, heads, kv, size, page = 21, 8, 4, 64, 8
    one = torch.randint(-20000, 20000, (3, rows, 1, size), dtype=torch.int16, device="cuda")
    row = torch.randint(-20000, 20000, (1, kv, size), dtype=torch.int16, device="cuda")
    freqs = torch.from_numpy(freqs_table(60, 48)).cuda()
    at = torch.arange(rows, dtype=torch.int32, device="cuda") * 2
    offsets = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    table = torch.arange(3, dtype=torch.int32, device="cuda").view(1, 3)
    results = []
    for write_out in (False, True):
        cache = torch.zeros(3, 2, page, kv * size, dtype=torch.int16, device="cuda")
        desc = pkm.PagedCache(data=cache, page_table=table, layer_stride=0, page_stride=cache.stride(0),
                              kv_stride=cache.stride(1), slot_stride=cache.stride(2), num_layers=1, num_pages=3,
                              page_size=page, row_elems=kv * size,
                              cache_lengths=torch.zeros(1, dtype=torch.int32, device="cuda"))
        q, k, v = one[0].expand(rows, heads, size), one[1].expand(rows, kv, size), row.expand(rows, kv, size)
        if write_out:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        out = torch.zeros(rows, heads, size, dtype=torch.int16, device="cuda")
        pkm.kv_rope_paged(offsets, at, freqs, desc, 0, kv, q=q, q_out=out, k=k, v=v, half=half)
        results.append((out, cache))
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
    assert results[0][0].any() and results[0][1].any()


def test_requests_on_the_same_pages():
    """A common beginning, and one request twice."""
    p = make_kv(38, [100, 100, 64], [20, 20, 40], 8, 2, 128, 16)
    p.table[1] = p.table[0]
    p.table[2, :4] = p.table[0, :4]
    p.q[20:40] = p.q[:20]
    d = check(p)
    assert torch.equal(d.out[:20], d.out[20:40]) and torch.equal(d.lse[:20], d.lse[20:40])


def test_orders_of_queries_and_outputs():
    """Queries with rows inside heads, and an output that starts 16 bytes into a sector."""
    p = make_kv(39, [300, 5], [1, 70], 6, 2, 128, 16)
    d = DeviceKv(p)
    d.run()
    torch.cuda.synchronize()
    first, lse = d.out.clone(), d.lse.clone()
    d.q = d.q.transpose(0, 1).contiguous().transpose(0, 1)
    assert d.q.stride(1) > d.q.stride(0)
    raw = torch.full((d.out.numel() + 16,), OUT_FILL, dtype=torch.int16, device="cuda")
    shifted = raw[8:8 + d.out.numel()].view(d.out.shape)
    assert shifted.data_ptr() % 32 == 16
    d.lse.fill_(LSE_FILL)
    d.run(out=shifted)
    torch.cuda.synchronize()
    assert torch.equal(shifted, first) and torch.equal(d.lse, lse)
    assert (raw[:8] == OUT_FILL).all() and (raw[-8:] == OUT_FILL).all()
    assert_kv_close(p, first.cpu().numpy().view(np.uint16), lse.cpu().numpy())


def test_keys_that_are_not_finite():
    """An attended NaN among the keys makes a row NaN, for the heads that share it; the rows that do
    not attend it are right."""
    p = make_kv(40, [100], [60], 4, 2, 64, 16)
    clean = p.reference()
    p.cache[p.layer, p.table[0, 130 // 16], 0, 130 % 16, 5] = 0x7FC0
    d = DeviceKv(p)
    d.run()
    out, lse, status = d.results()
    assert status == 0
    assert_kv_close(p, out, lse, clean, rows=np.arange(30))
    assert np.isnan(bf16_value(out[30:60, :2])).all() and np.isnan(lse[30:60, :2]).all()
    assert np.isfinite(bf16_value(out[:60, 2:])).all()
