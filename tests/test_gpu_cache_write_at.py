"""GPU: the cache write with rotary positions given apart from the slots.  With the rows' own
positions it writes mla_cache_write_paged's bits; with others, the bits of a row written where
that position is its own."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import workloads
from gpu_util import DeviceCacheWrite, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_mla_gb300  # noqa: F401


def write_at(g, positions, freqs=None, check=True):
    import paged_kv_mla_gb300 as pkm
    c = g.c
    f = g.freqs if freqs is None else freqs
    p = dev(positions.astype(np.uint32))
    if c.quantised:
        return pkm.mla_cache_write_paged_qcache_at(g.latent, g.iro, p, g.gamma, c.epsilon, f, g.qc,
                                                   c.layer_idx, dev_status=g.status, check=check)
    return pkm.mla_cache_write_paged_at(g.latent, g.iro, p, g.gamma, c.epsilon, f, g.pc, c.layer_idx,
                                        c.kv_lora_rank, c.rope_dim, dev_status=g.status, check=check)


def own_positions(c):
    iro = np.asarray(c.input_row_offsets, np.int64)
    out = np.zeros(c.latent.shape[0], np.int64)
    for b in range(len(iro) - 1):
        out[iro[b]:iro[b + 1]] = int(c.cache_lengths[b]) + np.arange(iro[b + 1] - iro[b])
    return out


CASES = [([7, 1, 300, 0, 45], [5, 0, 17, 3, 128], 512, 64, 16), ([1], [0], 128, 8, 4),
         ([33, 2], [0, 5], 256, 24, 64), ([64, 70, 3], [9, 2, 200], 512, 64, 128)]


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("new,lens,R,P,ps", CASES)
def test_own_positions_give_the_same_bits(new, lens, R, P, ps, quantised):
    c = workloads.make_cache_write("at", 900 + R + ps, new, lens, R, P, ps, num_layers=2,
                                   layer_idx=1, quantised=quantised)
    a, b = DeviceCacheWrite(c), DeviceCacheWrite(c)
    a.run()
    write_at(b, own_positions(c))
    x, y = a.results(), b.results()
    assert x[1] == y[1] == 0 and np.array_equal(x[0], y[0])


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("new,lens,R,P,ps", CASES)
def test_given_positions(new, lens, R, P, ps, quantised):
    """Random positions, with repeats: the same as writing with a table whose rows are
    permuted so that each row's own position holds the factors of the given one."""
    c = workloads.make_cache_write("at", 950 + R + ps, new, lens, R, P, ps, num_layers=2,
                                   layer_idx=1, quantised=quantised)
    gen = np.random.default_rng(R + ps)
    own = own_positions(c)
    seq = c.freqs_cis.shape[0]
    given = gen.integers(0, seq, len(own))
    for r0, r1 in zip(c.input_row_offsets[:-1], c.input_row_offsets[1:]):
        given[r0:r1] = np.where(gen.random(r1 - r0) < 0.5, own[r0:r1] // 2, given[r0:r1])
    b = DeviceCacheWrite(c)
    write_at(b, given)
    got, status = b.results()
    assert status == 0
    # one request at a time: its rows' own positions are distinct, so a table can serve them
    want = np.array(c.cache)
    for k in range(len(new)):
        r0, r1 = int(c.input_row_offsets[k]), int(c.input_row_offsets[k + 1])
        if r0 == r1:
            continue
        table = np.array(c.freqs_cis)
        table[own[r0:r1]] = c.freqs_cis[given[r0:r1]]
        a = DeviceCacheWrite(c)
        a.freqs = torch.from_numpy(table).cuda()
        a.run()
        one, _ = a.results()
        page = c.page_table[k][own[r0:r1] // ps]
        want[1, page, own[r0:r1] % ps] = one[1, page, own[r0:r1] % ps]
    assert np.array_equal(got, want)


def test_position_past_the_table_leaves_its_slot():
    c = workloads.make_cache_write("at", 990, [40], [3], 128, 16, 16)
    given = own_positions(c)
    given[[5, 39]] = [c.freqs_cis.shape[0], 0xFFFFFFFF]
    a, b = DeviceCacheWrite(c), DeviceCacheWrite(c)
    a.run()
    write_at(b, given)
    want, _ = a.results()
    got, status = b.results()
    assert status == 4
    for r in (5, 39):
        t = 3 + r
        at = (c.layer_idx, c.page_table[0][t // 16], t % 16)
        want[at] = c.cache[at]
    assert np.array_equal(got, want)
