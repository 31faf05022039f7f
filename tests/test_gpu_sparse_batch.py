"""GPU: a few rows among many requests without any, as of a batch padded to its largest size."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_mla_gb300  # noqa: F401


class Sparse:
    """`rows` requests of one row each, spread among `batch`; a page of its own for each."""

    def __init__(self, batch, rows, seed):
        import paged_kv_mla_gb300 as pkm
        gen = np.random.default_rng(seed)
        at = np.sort(gen.permutation(batch)[:rows])
        counts = np.zeros(batch, np.int64)
        counts[at] = 1
        self.at, self.rows, self.page = at, rows, 8
        self.lengths = gen.integers(0, 8, batch).astype(np.uint32)
        table = np.zeros((batch, 1), np.uint32)
        table[at, 0] = gen.permutation(rows)
        self.table = table
        self.latent = torch.randn(rows, 576, device="cuda").bfloat16()
        self.offsets = dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.uint32))
        self.gamma, self.freqs = torch.ones(512, device="cuda"), torch.randn(8, 64, device="cuda")
        self.data = torch.full((rows, 8, 576), -1, dtype=torch.int16, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cache = pkm.PagedCache(
            data=self.data, page_table=dev(table), layer_stride=rows * 8 * 576, page_stride=8 * 576,
            slot_stride=576, num_layers=1, num_pages=rows, page_size=8, row_elems=576,
            cache_lengths=dev(self.lengths))
        self.positions = dev(self.lengths[at])

    def run(self, at):
        import paged_kv_mla_gb300 as pkm
        a = (self.gamma, 1e-6, self.freqs, self.cache, 0, 512, 64)
        if at:
            pkm.mla_cache_write_paged_at(self.latent, self.offsets, self.positions, *a,
                                         dev_status=self.status)
        else:
            pkm.mla_cache_write_paged(self.latent, self.offsets, *a, dev_status=self.status)


@pytest.mark.parametrize("at", [False, True])
@pytest.mark.parametrize("batch,rows", [(33, 30), (70, 2), (1000, 30), (1000, 91), (30000, 30),
                                        (30000, 400)])
def test_rows_find_their_requests(batch, rows, at):
    s = Sparse(batch, rows, batch + rows)
    s.run(at)
    assert s.status.item() == 0
    got = s.data.view(torch.bfloat16).double().cpu().numpy()
    x = s.latent.double().cpu().numpy()
    nope = x[:, :512] / np.sqrt((x[:, :512] ** 2).mean(1, keepdims=True) + 1e-6)
    f = s.freqs.double().cpu().numpy()[s.lengths[s.at]]
    c, si, a, b = f[:, 0::2], f[:, 1::2], x[:, 512::2], x[:, 513::2]
    want = np.concatenate([nope, np.stack([a * c - b * si, a * si + b * c], -1).reshape(rows, 64)], 1)
    size = np.concatenate([np.abs(nope), np.repeat(np.abs(a * c) + np.abs(b * si), 2, 1) * 2
                           + np.repeat(np.abs(a * si) + np.abs(b * c), 2, 1)], 1)
    mine = got[s.table[s.at, 0], s.lengths[s.at]]
    # half a step of bf16, and a few fp32 roundings of the terms
    assert (np.abs(mine - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size).all()
    stay = np.ones(got.shape[:2], bool)
    stay[s.table[s.at, 0], s.lengths[s.at]] = False
    assert (s.data.cpu().numpy()[stay] == -1).all()


def test_time_does_not_grow_with_the_empty_requests():
    """A search takes as many steps as the logarithm of the requests; one request after the other
    takes 50 cycles and more for each of 30000: 0.7 ms at 2 GHz."""
    s = Sparse(30000, 30, 5)
    for _ in range(3):
        s.run(True)
    times = []
    for _ in range(10):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        s.run(True)
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    assert sorted(times)[5] < 200, times
