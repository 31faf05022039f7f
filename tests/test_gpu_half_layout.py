"""GPU: queries and keys in the half layout: the latent rows' rope columns turned like a head of
the queries, written with factors (1, 0), and attended."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from spec_util import (DeviceTree, assert_tree_close, bf16_bits, bf16_value, freqs_table, make_tree,
                       rotate64)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_mla_gb300  # noqa: F401


@pytest.mark.parametrize("at", [False, True])
def test_keys_and_queries_in_the_half_layout(at):
    import paged_kv_mla_gb300 as pkm
    from gpu_util import dev
    R, P, heads = 128, 32, 5
    p = make_tree(790, [0, 0], [40, 17], heads, R, P, page=16, tree=False)
    g = DeviceTree(p)
    g.cache.fill_(-1)  # what the writes below put there is all
    gen = np.random.default_rng(791)
    rows = p.rows
    bits = bf16_bits(gen.standard_normal((rows, R + P)))
    table = freqs_table(64, P)
    pos = np.concatenate([np.arange(40), np.arange(17)]).astype(np.uint32)
    latent, positions, f = dev(bits), dev(pos), torch.from_numpy(table).cuda()
    still = torch.zeros(64, P, device="cuda")
    still[:, 0::2] = 1
    keys = latent[:, None, R:]
    pkm.mla_rope_heads(keys, positions, f, keys, half=True, dev_status=g.status)
    a = (torch.ones(R, device="cuda"), 1e-6, still, g.desc, p.layer, R, P)
    if at:
        pkm.mla_cache_write_paged_at(latent, g.offsets, positions, *a, dev_status=g.status)
    else:
        pkm.mla_cache_write_paged(latent, g.offsets, *a, dev_status=g.status)
    q = g.q[..., R:]
    pkm.mla_rope_heads(q, positions, f, q, half=True, dev_status=g.status)
    g.run()
    out, lse, status = g.results()
    assert status == 0
    # the cache holds the turned keys, rounded once: half a step of bf16 and the products' fp32
    cells = g.cache.cpu().numpy().view(np.uint16)[p.layer]
    x = bf16_value(bits[:, R:])
    want = rotate64(x, table[pos].astype(np.float64), True)
    slots = np.concatenate([np.stack([p.table[b, t // 16], t % 16], 1) for b, n in ((0, 40), (1, 17))
                            for t in [np.arange(n)]])
    got = bf16_value(cells[slots[:, 0], slots[:, 1], R:R + P])
    size = np.abs(x).max(1, keepdims=True)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * size).all()
    turned = bf16_value(g.q.cpu().numpy().view(np.uint16)[..., R:])
    xq = bf16_value(p.q[..., R:])
    wq = rotate64(xq, table[pos].astype(np.float64)[:, None], True)
    assert (np.abs(turned - wq) <= 2.0 ** -8 * np.abs(wq) + 2.0 ** -21 * np.abs(xq).max()).all()
    # and the attention is that of the queries and keys as they now are
    p.q, p.cache = g.q.cpu().numpy().view(np.uint16), g.cache.cpu().numpy().view(np.uint16)
    assert_tree_close(p, out, lse)
