"""GPU: attention of new tokens (one, a chain, a drafted tree) over the paged latent cache
against the definition in 64 bits.  The tolerances are derived in spec_util.TreeProblem."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from spec_util import (LSE_FILL, OUT_FILL, DeviceTree, assert_tree_close, bf16_value, make_tree)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_mla_gb300  # noqa: F401  (raises if the library is missing)


def check(p):
    g = DeviceTree(p)
    g.run()
    out, lse, status = g.results()
    assert status == 0
    assert_tree_close(p, out, lse)
    return out, lse


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("ctx", [0, 1, 7, 63, 64, 127, 128, 129, 255, 256, 600])
def test_single_token(ctx, quantised):
    """One new token a request: the whole history and itself."""
    check(make_tree(100 + ctx, [ctx], [1], 16, page=64, tree=False, quantised=quantised))


@pytest.mark.parametrize("heads", [1, 3, 16, 20, 64, 96, 128, 130])
def test_head_counts(heads):
    check(make_tree(200 + heads, [200, 31], [3, 2], heads, page=16, tree=True))


@pytest.mark.parametrize("page", [1, 4, 8, 12, 16, 24, 32, 40, 64, 96, 128, 256])
@pytest.mark.parametrize("quantised", [False, True])
def test_page_sizes(page, quantised):
    """Pages that end inside, at and beyond the key tiles; sizes that are no multiple of 8."""
    check(make_tree(300 + page, [150, 5, 300], [4, 9, 1], 8, page=page, quantised=quantised))


@pytest.mark.parametrize("rank,rope", [(64, 16), (64, 0), (128, 32), (192, 64), (256, 64),
                                       (320, 8), (384, 192), (448, 128), (512, 0), (512, 24)])
def test_widths(rank, rope):
    check(make_tree(400 + rank + rope, [140, 12], [5, 3], 6, rank, rope, page=32))


@pytest.mark.parametrize("rank,rope", [(128, 64), (256, 0), (384, 48), (512, 64)])
def test_quantised_widths(rank, rope):
    check(make_tree(450 + rank + rope, [140, 12], [5, 3], 6, rank, rope, page=32, quantised=True))


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("new", [2, 31, 32, 33, 64, 65, 130])
def test_tree_sizes(new, tree):
    """Masks that end inside, at and beyond a word; drafts over several key tiles."""
    check(make_tree(500 + new, [77], [new], 4, page=16, tree=tree))


@pytest.mark.parametrize("quantised", [False, True])
def test_ragged_batch(quantised):
    ctx = [0, 5, 128, 1000, 64, 0, 333, 17, 90]
    new = [1, 0, 23, 2, 64, 7, 0, 1, 12]
    check(make_tree(600, ctx, new, 16, page=16, quantised=quantised))


def test_many_requests():
    gen = np.random.default_rng(3)
    ctx = [int(x) for x in gen.integers(0, 90, 400)]
    new = [int(x) for x in gen.integers(0, 3, 400)]
    check(make_tree(601, ctx, new, 2, 128, 16, page=8))


def test_long_history_is_split():
    """Every pair of CTAs takes a part of one request's keys."""
    check(make_tree(602, [20011], [2], 16, 512, 64, page=64))


def test_padded_slots_and_strides():
    check(make_tree(603, [100, 40], [3, 5], 5, 256, 64, page=16, pad=16))
    check(make_tree(604, [100, 40], [3, 5], 5, 256, 64, page=16, pad=48, quantised=True))


def test_rows_that_attend_nothing():
    """No history and an empty mask row: zeros and lse = -inf; its neighbours are unaffected."""
    bits = [1, 0, 0b101, 0, 0, 1]
    p = make_tree(605, [0, 0, 30], [4, 1, 1], 7, bits=bits)
    out, lse = check(p)
    for r in (1, 3, 4):
        assert not out[r].any() and np.isneginf(lse[r]).all()
    assert np.isfinite(lse[5]).all()


def test_mask_bits_beyond_the_request():
    """Set bits behind the request's last token, and tokens behind the mask's last word."""
    p = make_tree(606, [20, 9], [3, 40], 4, words=1, bits=[0xFFFFFFFF] * 43)
    check(p)


def test_masked_rows_may_hold_nan_and_infinity():
    """What a row does not attend leaves its result as it is, bit for bit."""
    p = make_tree(607, [50], [6], 16, bits=[1, 3, 5, 9, 17, 33])
    a = DeviceTree(p)
    a.run()
    out0, lse0, _ = a.results()
    for j, v in ((2, 0x7FC0), (4, 0x7F80), (5, 0xFF80)):
        t = p.ctx[0] + j
        p.cache[p.layer, p.table[0][t // p.page], t % p.page] = v
    b = DeviceTree(p)
    b.run()
    out1, lse1, status = b.results()
    assert status == 0
    for r in (0, 1, 3):
        assert np.array_equal(out0[r], out1[r]) and np.array_equal(lse0[r], lse1[r])
    assert np.isnan(bf16_value(out1[2])).all()  # token 2 attends its own NaN row


def test_masked_quantised_rows_may_hold_nan():
    p = make_tree(608, [50], [4], 16, bits=[1, 3, 5, 9], quantised=True)
    a = DeviceTree(p)
    a.run()
    out0, lse0, _ = a.results()
    t = p.ctx[0] + 2
    p.cache[p.layer, p.table[0][t // p.page], t % p.page] = 0xFF
    b = DeviceTree(p)
    b.run()
    out1, lse1, _ = b.results()
    for r in (0, 1, 3):
        assert np.array_equal(out0[r], out1[r]) and np.array_equal(lse0[r], lse1[r])


def test_rows_outside_the_requests_stay():
    """Offsets that start above zero and end before total_rows."""
    p = make_tree(609, [33, 4], [3, 2], 5)
    p.q = np.concatenate([p.q, p.q], 0)[:9]
    p.mask = np.concatenate([p.mask, p.mask], 0)[:9]
    p.offsets = p.offsets + 2
    g = DeviceTree(p)
    g.run()
    out, lse, status = g.results()
    assert status == 0
    for r in (0, 1, 7, 8):
        assert (out[r] == OUT_FILL).all() and (lse[r] == LSE_FILL).all()
    ref = p.reference()
    rows = slice(2, 7)
    assert (np.abs(bf16_value(out[rows]) - ref[0][rows]) <= ref[1][rows]).all()


@pytest.mark.parametrize("q_std,scale", [(30.0, None), (0.0, None), (1.0, 0.0), (1.0, -0.5),
                                         (1.0, 3.0)])
def test_score_ranges(q_std, scale):
    """Scores far apart (one weight near 1), all equal, and negative scales."""
    p = make_tree(610, [300, 70], [2, 5], 8, 256, 64, q_std=q_std, scale=scale)
    g = DeviceTree(p)
    g.run()
    out, lse, status = g.results()
    assert status == 0
    assert_tree_close(p, out, lse)


def test_growing_scores():
    """Keys whose scores keep growing along the history: the running maximum moves on."""
    p = make_tree(611, [1500], [1], 4, 128, 0, page=32, tree=False)
    t = np.arange(1500)
    rows = bf16_value(p.cache[p.layer, p.table[0][t // 32], t % 32])
    from spec_util import bf16_bits
    direction = bf16_value(p.q[0, 0])
    rows = rows + np.outer(t / 15.0, direction) / np.linalg.norm(direction)
    p.cache[p.layer, p.table[0][t // 32], t % 32] = bf16_bits(rows)
    check(p)


def test_without_lse_and_repeatable():
    p = make_tree(612, [3000, 700], [2, 9], 16, 512, 64, page=64)
    g = DeviceTree(p)
    g.run()
    out0, lse0, _ = g.results()
    g.out.fill_(0)
    g.workspace = g.new_workspace()
    g.run(lse=False)
    out1, _, status = g.results()
    assert status == 0 and np.array_equal(out0, out1)
    for _ in range(3):
        g.run()
    out2, lse2, _ = g.results()
    assert np.array_equal(out0, out2) and np.array_equal(lse0, lse2)


def test_out_of_range_tokens_are_reported():
    """A page id past the cache and a history past the page-table row: reported, the other
    request's rows as they would be."""
    p = make_tree(613, [100, 60, 40], [1, 2, 2], 4, page=16)
    ref = p.reference()
    p.table[0, 3] = 0x40000000
    g = DeviceTree(p)
    g.lengths[2] = 100000
    g.run()
    out, lse, status = g.results()
    assert status == 4
    assert (np.abs(bf16_value(out[1:3]) - ref[0][1:3]) <= ref[1][1:3]).all()


def test_other_stream_and_graph():
    p = make_tree(614, [900, 20], [4, 3], 16, 512, 64, page=64)
    g = DeviceTree(p)
    ref = p.reference()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g.run(stream=s)
    s.synchronize()
    out, lse, status = g.results()
    assert status == 0
    assert_tree_close(p, out, lse, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.run()
    # the replay follows the device arrays: shorter histories, other queries
    g.out.fill_(0)
    graph.replay()
    again, lse2, _ = g.results()
    assert np.array_equal(out, again) and np.array_equal(lse, lse2)
    p2 = make_tree(614, [900, 20], [4, 3], 16, 512, 64, page=64)
    p2.ctx = [500, 20]
    t = np.arange(4)
    for j in t:  # request 0's drafts now follow token 499
        src, dst = 900 + j, 500 + j
        p2.cache[1, p2.table[0][dst // 64], dst % 64] = p2.cache[1, p2.table[0][src // 64], src % 64]
    g.cache.copy_(torch.from_numpy(p2.cache.view(np.int16)))
    g.lengths[0] = 500
    graph.replay()
    out, lse, status = g.results()
    assert status == 0
    assert_tree_close(p2, out, lse)


def test_two_calls_at_once():
    """Two streams, a workspace each."""
    a, b = (DeviceTree(make_tree(615 + k, [2500, 40], [3, 5], 16, 256, 64, page=32)) for k in (0, 1))
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for x in (s, t):
        x.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        a.run(stream=s)
        b.run(stream=t)
    for g in (a, b):
        out, lse, status = g.results()
        assert status == 0
        assert_tree_close(g.p, out, lse)


def test_cache_beyond_32_bit_offsets():
    """A layer of more than 2^32 bytes: rows at its far end."""
    p = make_tree(617, [70, 200], [2, 3], 4, 512, 64, page=64, layers=1, layer=0)
    g = DeviceTree(p)
    L, N, S, E = p.cache.shape
    stride = 1 << 29  # elements between pages: page 4 starts beyond 2^32 bytes
    big = torch.full(((N - 1) * stride + S * E,), 0x7FC0, dtype=torch.int16, device="cuda")
    for k in range(N):
        big[k * stride:k * stride + S * E] = g.cache[0, k].flatten()
    g.desc.data, g.desc.page_stride, g.desc.layer_stride = big, stride, 0
    g.run()
    out, lse, status = g.results()
    assert status == 0
    assert_tree_close(p, out, lse)


@pytest.mark.parametrize("page", [128, 256, 64])
def test_drafts_over_tiles_of_many_items(page):
    """Several 128-row items per pair of CTAs whose drafts lie in one or two key tiles, pages
    of whole tiles: the value buffers change their use from item to item."""
    gen = np.random.default_rng(page)
    ctx = [int(x) for x in gen.integers(0, 400, 40)]
    new = [int(x) for x in gen.integers(1, 65, 40)]
    check(make_tree(620 + page, ctx, new, 24, 512, 64, page=page))


@pytest.mark.parametrize("rank,rope", [(64, 16), (64, 0), (128, 32), (192, 64), (256, 64),
                                       (320, 8), (384, 192), (448, 128), (512, 0), (512, 24),
                                       (512, 64)])
def test_widths_of_rows_by_loads(rank, rope):
    """Pages of no multiple of 8 slots."""
    check(make_tree(630 + rank + rope, [140, 300], [5, 3], 6, rank, rope, page=12))


@pytest.mark.parametrize("new", [1, 33, 65, 130, 260])
@pytest.mark.parametrize("page,quantised", [(12, False), (64, True), (64, False)])
def test_drafts_over_several_tiles(new, page, quantised):
    check(make_tree(640 + new, [77, 0, 300], [new, 2, 5], 4, page=page, quantised=quantised))


@pytest.mark.parametrize("page,quantised", [(12, False), (32, True), (32, False)])
def test_falling_and_growing_scores(page, quantised):
    """Scores that grow towards one end of the history, from which the maximum moves on."""
    p = make_tree(650, [1500], [1], 4, 512, 64, page=page, tree=False, quantised=quantised)
    p.q[:, 1] = p.q[:, 0] ^ 0x8000  # head 1: minus head 0's, so one grows where the other falls
    from spec_util import bf16_bits
    t = np.arange(1500)
    c = 512 if quantised else 0  # the rope columns are bf16 in both
    cells = p.cache[p.layer, p.table[0][t // page], t % page]
    rope = cells[:, 512:512 + 128].copy().view(np.uint16) if quantised else cells[:, 512:576]
    direction = bf16_value(p.q[0, 0, 512:])
    rows = bf16_value(rope) + np.outer(t / 20.0, direction) / np.linalg.norm(direction)
    bits = bf16_bits(rows)
    cells[:, c if quantised else 512:c + 128 if quantised else 576] = \
        bits.view(np.uint8) if quantised else bits
    p.cache[p.layer, p.table[0][t // page], t % page] = cells
    check(p)


def test_output_between_sectors():
    """An output that is 16-byte but not 32-byte aligned."""
    p = make_tree(651, [100, 9], [40, 3], 8, 512, 64, page=64)
    g = DeviceTree(p)
    flat = torch.full((g.out.numel() + 8,), OUT_FILL, dtype=torch.int16, device="cuda")
    g.out = flat[8:].view(g.out.shape)
    assert g.out.data_ptr() % 32 == 16
    g.run()
    out, lse, status = g.results()
    assert status == 0 and (flat[:8] == flat[0]).all()
    assert_tree_close(p, out, lse)


@pytest.mark.parametrize("page,quantised", [(100, False), (64, True)])
def test_rows_by_loads_beyond_32_bit_offsets(page, quantised):
    p = make_tree(652, [70, 200], [2, 3], 4, 512, 64, page=page, layers=1, layer=0,
                  quantised=quantised)
    g = DeviceTree(p)
    L, N, S, E = p.cache.shape
    stride = 1 << 30 if quantised else 1 << 29  # pages a GiB apart
    big = torch.full(((N - 1) * stride + S * E,), 0x7F, dtype=g.cache.dtype, device="cuda")
    for k in range(N):
        big[k * stride:k * stride + S * E] = g.cache[0, k].flatten()
    g.desc.data, g.desc.page_stride, g.desc.layer_stride = big, stride, 0
    g.run()
    out, lse, status = g.results()
    assert status == 0
    assert_tree_close(p, out, lse)


def test_one_page_without_a_stride():
    """A cache of a single page, whose page stride says nothing."""
    for quantised in (False, True):
        p = make_tree(653, [100], [3], 4, 512, 64, page=128, layers=1, layer=0, quantised=quantised)
        used = int(p.table[0, 0])
        p.cache = p.cache[:, used:used + 1].copy()
        p.table = np.zeros_like(p.table[:, :1])
        g = DeviceTree(p)
        g.desc.page_stride = 0
        g.run()
        out, lse, status = g.results()
        assert status == 0
        assert_tree_close(p, out, lse)


def test_refuses_views_and_host_memory():
    import paged_kv_mla_gb300 as pkm
    p = make_tree(654, [20], [3], 4, 512, 64, page=64)
    g = DeviceTree(p)
    args = dict(tree_mask=g.mask, lse=g.lse, check=False)

    def call(q=g.q, out=g.out, **kw):
        return pkm.mla_tree_attention_paged(q, g.offsets, p.scale, g.desc, p.layer, 512, 64, out,
                                            g.workspace, **{**args, **kw})
    assert call() == 0
    assert call(q=g.q.cpu()) == 1
    assert call(out=torch.zeros(3, 4, 576, dtype=torch.int16, device="cuda")[:, :, :512]) == 1
    assert call(tree_mask=g.mask.long()) == 1
    assert call(lse=g.lse.double()) == 1
    torch.cuda.synchronize()


@pytest.mark.parametrize("page,quantised", [(12, False), (16, True), (64, False)])
def test_out_of_range_tokens_by_every_source(page, quantised):
    """Page ids that the cache does not have and a history past the table's row, by loads, from
    quantised rows and by wide boxes: reported, and the other requests' rows as they would be."""
    p = make_tree(655, [100, 300, 40], [1, 2, 2], 4, 512, 64, page=page, quantised=quantised)
    ref = p.reference()
    p.table[0, 0] = 0x40000000
    g = DeviceTree(p)
    g.lengths[2] = 100000
    g.run()
    out, lse, status = g.results()
    assert status == 4
    assert (np.abs(bf16_value(out[1:3]) - ref[0][1:3]) <= ref[1][1:3]).all()
