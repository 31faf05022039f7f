"""GPU: compaction of accepted drafts against a copy loop on the host, bit for bit over the
whole cache."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import dev
from spec_util import page_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_mla_gb300  # noqa: F401


class Problem:
    """ctx, drafts and accepted paths; cache [layers, planes, pages, page, slot] of random bits."""

    def __init__(self, seed, ctx, new, paths, page, rank=512, rope=64, quantised=False, layers=3,
                 planes=1, pad=16, width=None):
        gen = np.random.default_rng(seed)
        self.ctx, self.paths, self.page, self.planes = ctx, paths, page, planes
        self.table, pages = page_table(gen, ctx, new, page)
        self.quantised = quantised
        self.rank, self.rope = rank, rope
        if quantised:
            self.payload = rank + 2 * rope + rank // 32
            slot = (self.payload + 15) // 16 * 16 + pad
            self.cache = gen.integers(0, 256, (layers, planes, pages, page, slot), dtype=np.uint8)
        else:
            self.payload = rank + rope
            self.cache = gen.integers(0, 65536, (layers, planes, pages, page, self.payload + pad),
                                      dtype=np.uint16)
        self.width = width or max(1, max(len(p) for p in paths))
        self.accepted = np.full((len(ctx), self.width), 0xFFFFFFFF, np.uint32)
        for b, p in enumerate(paths):
            self.accepted[b, :len(p)] = p
        self.counts = np.array([len(p) for p in paths], np.uint32)

    def run(self, begin=0, count=None, graph=False):
        import paged_kv_mla_gb300 as pkm
        L, V, N, S, E = self.cache.shape
        count = L - begin if count is None else count
        data, table = dev(self.cache), dev(self.table)
        lengths = dev(np.asarray(self.ctx, np.uint32))
        sizes = dict(data=data, page_table=table, layer_stride=V * N * S * E, page_stride=S * E,
                     slot_stride=E, num_layers=L, num_pages=N, page_size=S, cache_lengths=lengths)
        acc, counts = dev(self.accepted), dev(self.counts)
        out = torch.full((len(self.ctx),), -7, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        if self.quantised:
            c = pkm.QuantCache(kv_lora_rank=self.rank, rope_dim=self.rope, **sizes)
            call = pkm.mla_cache_compact_paged_qcache
        else:
            c = pkm.PagedCache(row_elems=self.payload, kv_stride=N * S * E if V == 2 else 0, **sizes)
            call = pkm.mla_cache_compact_paged
        if graph:
            start = data.clone()
            call(c, begin, count, acc, counts, out, dev_status=status)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call(c, begin, count, acc, counts, out, dev_status=status)
            data.copy_(start)
            out.fill_(-7)
            g.replay()
        else:
            call(c, begin, count, acc, counts, out, dev_status=status)
        torch.cuda.synchronize()
        return (data.cpu().numpy().view(self.cache.dtype).reshape(self.cache.shape),
                out.cpu().numpy(), int(status.item()))

    def expected(self, begin=0, count=None, skip=()):
        want = self.cache.copy()
        L = self.cache.shape[0]
        lengths = []
        for b, path in enumerate(self.paths):
            lengths.append(self.ctx[b] + (0 if b in skip else len(path)))
            if b in skip:
                continue
            at = lambda t: (self.table[b][t // self.page], t % self.page)
            for l in range(begin, L if count is None else begin + count):
                for v in range(self.planes):
                    for j, t in enumerate(path):
                        want[l, v][at(self.ctx[b] + j)][:self.payload] = \
                            self.cache[l, v][at(self.ctx[b] + t)][:self.payload]
        return want, np.array(lengths)


PATHS = [[0], [], [0, 1, 2], [1, 2, 3, 4], [0, 5, 9], [3], list(range(1, 64, 2)), [2, 63],
         list(range(64))]


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("page", [1, 8, 12, 64, 128])
def test_paths(page, quantised):
    """Overlapping moves (every row the next one's source), no moves, no accepted drafts."""
    ctx = [0, 5, 63, 64, 100, 17, 1, 200, 31]
    p = Problem(page, ctx, [64] * 9, PATHS, page, quantised=quantised)
    got, lengths, status = p.run()
    want, want_lengths = p.expected()
    assert status == 0 and np.array_equal(lengths, want_lengths) and np.array_equal(got, want)


@pytest.mark.parametrize("rank,rope,quantised", [(64, 16, False), (8, 0, False), (1024, 256, False),
                                                 (128, 64, True), (128, 0, True), (384, 8, True),
                                                 (1024, 256, True)])
def test_widths(rank, rope, quantised):
    """Payloads that are no multiple of 16 bytes among the quantised ones."""
    p = Problem(rank + rope, [10, 20], [20, 9], [[1, 4, 19], [0, 2, 3, 8]], 16, rank, rope, quantised)
    got, lengths, status = p.run()
    want, want_lengths = p.expected()
    assert status == 0 and np.array_equal(lengths, want_lengths) and np.array_equal(got, want)


def test_long_path_over_several_tables():
    gen = np.random.default_rng(5)
    path = sorted(int(x) for x in gen.choice(700, 300, replace=False))
    p = Problem(6, [3], [700], [path], 32, 64, 16)
    got, lengths, status = p.run()
    want, want_lengths = p.expected()
    assert status == 0 and np.array_equal(lengths, want_lengths) and np.array_equal(got, want)


def test_two_planes_and_layer_range():
    p = Problem(7, [10, 3], [12, 12], [[0, 4, 11], [2, 3]], 16, 128, 0, layers=5, planes=2)
    got, lengths, status = p.run(begin=1, count=3)
    want, want_lengths = p.expected(begin=1, count=3)
    assert status == 0 and np.array_equal(lengths, want_lengths) and np.array_equal(got, want)


def test_invalid_requests_stay_as_they_are():
    """A count past the row, a repeated index, a decreasing one, a position past the table:
    reported, nothing moved, and the valid request beside them served."""
    paths = [[1, 2], [1, 2], [1, 2], [1, 2], [1, 5]]
    p = Problem(8, [10, 10, 10, 10, 4], [8] * 5, paths, 8, 64, 16)
    p.counts[0] = 3
    p.accepted[1] = [2, 2]
    p.accepted[2] = [4, 1]
    p.accepted[3] = [1, 100000]
    got, lengths, status = p.run()
    want, want_lengths = p.expected(skip=(0, 1, 2, 3))
    assert status == 4 and np.array_equal(lengths, want_lengths) and np.array_equal(got, want)
    p.accepted[3] = [1, 2]
    got, lengths, status = p.run()
    want, want_lengths = p.expected(skip=(0, 1, 2))
    assert status == 1 and np.array_equal(lengths, want_lengths) and np.array_equal(got, want)


def test_captured_and_replayed():
    p = Problem(9, [10, 3, 90], [30, 12, 4], [[0, 4, 11, 29], [2, 3], []], 16)
    got, lengths, status = p.run(graph=True)
    want, want_lengths = p.expected()
    assert status == 0 and np.array_equal(lengths, want_lengths) and np.array_equal(got, want)
