"""GPU: rotary positions on several axes and the write of keys and values, against the turn in 64
bits.  Two fp32 products and a sum of bf16 inputs, rounded once: off by at most half a bf16 step
(2^-8 of the value) and 2^-22 of the pair's size (three fp32 roundings, and cancellation)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import dev
from kv_util import LAYOUTS, device_cache
from spec_util import bf16_bits, bf16_value, freqs_table, page_table, rotate64

pytestmark = pytest.mark.gpu
FILL = 0x1234


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_mla_gb300  # noqa: F401


class Problem:
    def __init__(self, seed, ctx, new, heads, kv_heads, size, P, axes=3, seq=700, page=16, layout="page",
                 pad=0, pair_axes="runs"):
        gen = np.random.default_rng(seed)
        self.ctx, self.new, self.P, self.page, self.kv_heads, self.size = ctx, new, P, page, kv_heads, size
        self.rows = sum(new)
        self.table, pages = page_table(gen, ctx, new, page)
        row = kv_heads * size
        dims, order = (2, pages, 2, page), LAYOUTS[layout]
        store = np.full([dims[i] for i in order] + [row + pad], FILL, np.uint16)
        self.cache = store.transpose(*[order.index(i) for i in range(4)], 4)
        self.q, self.k, self.v = (bf16_bits(gen.standard_normal((self.rows, h, size)))
                                  for h in (heads, kv_heads, kv_heads))
        self.offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.uint32)
        self.positions = gen.integers(0, seq, (axes, self.rows)).astype(np.uint32)
        self.positions[0, :1] = seq - 1
        j = np.arange(P // 2)
        self.pair_axes = {"runs": j * axes // (P // 2), "turns": j % axes,
                          "last": 0 * j + axes - 1}[pair_axes].tolist()
        self.freqs = freqs_table(seq, P) * np.float32(1.25)

    def factors(self):
        f = self.freqs.astype(np.float64).reshape(len(self.freqs), -1, 2)
        j = np.arange(self.P // 2)
        return f[self.positions[self.pair_axes].T, j].reshape(self.rows, 1, self.P)

    def device(self):
        desc, cache = device_cache(self.cache, dev(self.table), dev(np.asarray(self.ctx, np.uint32)),
                                   self.kv_heads * self.size)
        return desc, cache, torch.from_numpy(self.freqs).cuda(), dev(self.positions), dev(self.offsets)

    def slots(self, r):
        b = int(np.searchsorted(self.offsets, r, side="right")) - 1
        t = self.ctx[b] + r - int(self.offsets[b])
        return self.table[b, t // self.page], t % self.page


def assert_turned(got, x, cs, P, half, rows=None):
    pick = slice(None) if rows is None else rows
    got, x, cs = got[pick], x[pick], cs[pick]
    assert np.array_equal(got[..., P:], x[..., P:])  # copied
    x64 = bf16_value(x[..., :P])
    ref = rotate64(x64, cs, half)
    size = rotate64(np.abs(x64), np.abs(cs) * np.where(np.arange(P) % 2, -1.0, 1.0), half)
    size = np.maximum(np.abs(size), np.abs(ref)) + np.abs(x64).max()
    assert (np.abs(bf16_value(got[..., :P]) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * size).all()


def run(p, half, q=True, k=True, v=True, layer=1, q_in=None, q_out=None):
    import paged_kv_mla_gb300 as pkm
    desc, cache, freqs, positions, offsets = p.device()
    q_in = dev(p.q) if q_in is None else q_in
    q_out = torch.full(p.q.shape, FILL, dtype=torch.int16, device="cuda") if q_out is None else q_out
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkm.kv_rope_paged(offsets, positions, freqs, desc, layer, p.kv_heads, q=q_in if q else None,
                      q_out=q_out if q else None, k=dev(p.k) if k else None, v=dev(p.v) if v else None,
                      pair_axes=p.pair_axes, half=half, dev_status=status)
    torch.cuda.synchronize()
    return q_out.cpu().numpy().view(np.uint16), cache.cpu().numpy().view(np.uint16), status.item()


def assert_cache(p, got, before, half, layer=1, keys=True, values=True, rows=None, key_rows=None):
    """The rows' slots hold turned keys and values; every other element is as it was."""
    cs, row = p.factors(), p.kv_heads * p.size
    rest = got.copy()
    for r in range(p.rows) if rows is None else rows:
        page, slot = p.slots(r)
        if keys:
            src = p.k[r] if key_rows is None else key_rows[r]
            assert_turned(got[layer, page, 0, slot, :row].reshape(1, p.kv_heads, p.size), src[None],
                          cs[r:r + 1], p.P, half)
            rest[layer, page, 0, slot, :row] = before[layer, page, 0, slot, :row]
        if values:
            assert np.array_equal(got[layer, page, 1, slot, :row], p.v[r].ravel())
            rest[layer, page, 1, slot, :row] = before[layer, page, 1, slot, :row]
    assert np.array_equal(rest, before)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("heads,kv_heads,size,P", [(1, 1, 8, 8), (32, 8, 128, 128), (16, 2, 64, 64),
                                                   (5, 1, 24, 16), (7, 7, 256, 256), (130, 2, 128, 64),
                                                   (12, 3, 104, 48), (2, 66, 16, 16)])
@pytest.mark.parametrize("axes,pair_axes", [(1, "runs"), (3, "runs"), (3, "turns"), (4, "turns"), (2, "last")])
def test_queries_keys_and_values(heads, kv_heads, size, P, axes, pair_axes, half):
    p = Problem(heads + size + axes, [40, 0, 15], [1, 20, 3], heads, kv_heads, size, P, axes, pair_axes=pair_axes)
    q, cache, status = run(p, half)
    assert status == 0
    assert_turned(q, p.q, p.factors(), P, half)
    assert_cache(p, cache, p.cache, half)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("layout", ["page", "plane", "slot"])
def test_strided_parts_of_one_projection(layout, half):
    import paged_kv_mla_gb300 as pkm
    p = Problem(3, [7, 100], [30, 11], 6, 2, 64, 32, layout=layout, pad=8, page=12)
    desc, cache, freqs, positions, offsets = p.device()
    x = torch.cat([dev(p.q), dev(p.k), dev(p.v)], 1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # the queries in place
    pkm.kv_rope_paged(offsets, positions, freqs, desc, 0, 2, q=x[:, :6], q_out=x[:, :6], k=x[:, 6:8], v=x[:, 8:],
                      pair_axes=p.pair_axes, half=half, dev_status=status)
    assert status.item() == 0
    got = x.cpu().numpy().view(np.uint16)
    assert_turned(got[:, :6], p.q, p.factors(), p.P, half)
    assert np.array_equal(got[:, 6:8], p.k) and np.array_equal(got[:, 8:], p.v)
    assert_cache(p, cache.cpu().numpy().view(np.uint16), p.cache, half, layer=0)


@pytest.mark.parametrize("half", [False, True])
def test_keys_in_place_as_the_projection_leaves_them(half):
    """Without k: what the slots hold turns; without v: the V plane stays; with and without q."""
    for q in (False, True):
        p = Problem(4, [3, 0, 31], [5, 0, 40], 8, 4, 128, 64, page=8)
        for r in range(p.rows):
            page, slot = p.slots(r)
            p.cache[1, page, 0, slot] = p.k[r].ravel()
        before = p.cache.copy()
        got_q, cache, status = run(p, half, q=q, k=False, v=False)
        assert status == 0
        if q:
            assert_turned(got_q, p.q, p.factors(), p.P, half)
        assert_cache(p, cache, before, half, values=False, key_rows=p.k)
    got_q, cache, status = run(p, half, k=False, v=True)
    assert_cache(p, cache, before, half, key_rows=p.k)


def test_one_axis_is_the_rotation_of_heads():
    """The same bits as mla_rope_heads, for positions of one dimension and without pair_axes."""
    import paged_kv_mla_gb300 as pkm
    p = Problem(5, [90], [50], 16, 2, 64, 64, axes=1)
    desc, cache, freqs, positions, offsets = p.device()
    a, b = torch.empty(2, 50, 16, 64, dtype=torch.int16, device="cuda")
    for half in (False, True):
        pkm.kv_rope_paged(offsets, positions[0], freqs, desc, 0, 2, q=dev(p.q), q_out=a, k=dev(p.k), half=half)
        pkm.mla_rope_heads(dev(p.q), positions[0], freqs, b, half=half)
        assert torch.equal(a, b)


def test_positions_and_slots_out_of_range():
    p = Problem(6, [10, 20], [12, 6], 4, 2, 64, 64, axes=3, seq=50, page=8)
    p.positions[1, 4] = 50
    p.positions[2, 9] = 0xFFFFFFFF
    p.table[1, 3] = 0x40000000  # positions 24, 25
    lost, unslotted = [4, 9], [16, 17]
    q, cache, status = run(p, True)
    assert status == 4
    keep = [r for r in range(p.rows) if r not in lost]
    p.positions[:, lost] = 0
    assert (q[lost] == FILL).all()
    assert_turned(q, p.q, p.factors(), p.P, True, rows=keep)
    assert_cache(p, cache, p.cache, True, rows=[r for r in keep if r not in unslotted])


def test_table_too_short_and_rows_outside_the_requests():
    import paged_kv_mla_gb300 as pkm
    p = Problem(7, [10], [12], 4, 2, 64, 64, axes=2, page=8)
    desc, cache, freqs, positions, offsets = p.device()
    desc.page_table = dev(p.table[:, :2])  # positions from 16 on have no page
    out = torch.full(p.q.shape, FILL, dtype=torch.int16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkm.kv_rope_paged(offsets, positions, freqs, desc, 1, 2, q=dev(p.q), q_out=out, k=dev(p.k), v=dev(p.v),
                      pair_axes=p.pair_axes, dev_status=status)
    assert status.item() == 4
    assert_cache(p, cache.cpu().numpy().view(np.uint16), p.cache, False, rows=range(6))
    # offsets [2, 9]: the request's tokens are rows 2 .. 8
    p = Problem(8, [10], [12], 4, 2, 64, 64, axes=2, page=8)
    desc, cache, freqs, positions, _ = p.device()
    out.fill_(FILL)
    pkm.kv_rope_paged(dev(np.array([2, 9], np.uint32)), positions, freqs, desc, 1, 2, q=dev(p.q), q_out=out,
                      k=dev(p.k), v=dev(p.v), pair_axes=p.pair_axes)
    got = out.cpu().numpy().view(np.uint16)
    assert (got[:2] == FILL).all() and (got[9:] == FILL).all()
    assert_turned(got, p.q, p.factors(), p.P, False, rows=list(range(2, 9)))
    p.ctx, p.offsets = [8], np.array([0, 12], np.uint32)  # row r at 10 + r - 2
    assert_cache(p, cache.cpu().numpy().view(np.uint16), p.cache, False, rows=range(2, 9))


def test_many_requests_some_empty():
    gen = np.random.default_rng(9)
    new = gen.integers(0, 3, 1500).tolist()
    p = Problem(9, gen.integers(0, 30, 1500).tolist(), new, 4, 1, 64, 64, page=16)
    q, cache, status = run(p, True)
    assert status == 0
    assert_turned(q, p.q, p.factors(), p.P, True)
    assert_cache(p, cache, p.cache, True)


def test_captured_and_replayed():
    import paged_kv_mla_gb300 as pkm
    p = Problem(10, [5, 60], [40, 10], 8, 2, 128, 128)
    desc, cache, freqs, positions, offsets = p.device()
    x = torch.cat([dev(p.q), dev(p.k), dev(p.v)], 1)
    out = torch.zeros(50, 8, 128, dtype=torch.int16, device="cuda")

    def call():
        pkm.kv_rope_paged(offsets, positions, freqs, desc, 1, 2, q=x[:, :8], q_out=out, k=x[:, 8:10], v=x[:, 10:],
                          pair_axes=p.pair_axes, half=True)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    p2 = Problem(11, [5, 60], [40, 10], 8, 2, 128, 128)
    p2.table = p.table
    x.copy_(torch.cat([dev(p2.q), dev(p2.k), dev(p2.v)], 1))
    positions.copy_(dev(p2.positions))
    graph.replay()
    torch.cuda.synchronize()
    assert_turned(out.cpu().numpy().view(np.uint16), p2.q, p2.factors(), 128, True)
    assert_cache(p2, cache.cpu().numpy().view(np.uint16), p.cache, True)
