"""GPU: where the line of all requests' key tiles is cut into the blocks' shares, at 33 million tiles.  A
tile that is left out, taken twice or taken from another place shows: some hold a key that outweighs
all ordinary ones together, so that one of it more or less moves the log-sum-exp by a tenth and more."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ITEM_COST = 2  # units that an item counts besides its tiles: where the cuts lie, not what is right


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_mla_gb300  # noqa: F401


@pytest.mark.parametrize("size", [64, 128])
def test_marked_tiles(size):
    """512 requests of 2^20 tokens, every page of theirs the same but the marked ones: tiles at both
    sides of each cut, some requests' first and last, and some anywhere."""
    import paged_kv_mla_gb300 as pkm
    n, heads, page, tiles, slot = 512, 8, 128, 8192, 77
    gen = torch.Generator(device="cuda").manual_seed(71)
    cache = torch.randn(2, 2, page, heads, size, device="cuda", generator=gen)
    q = torch.randn(n, heads, size, device="cuda", generator=gen)
    cache[1] = cache[0]
    cache[:, 0, :, :, 0] = 0.0
    q[:, :, 0] = 8.0
    scale = 0.125
    cache[1, 0, slot] = 0.0
    cache[1, 0, slot, :, 0] = 16.0  # a score of 16 for every query: exp(16) is 5 times 2^20 exp(1/2)
    cache[1, 1, slot] = 4.0
    cache, q = cache.bfloat16(), q.bfloat16()

    marks = np.zeros((n, tiles), bool)
    blocks = min(torch.cuda.get_device_properties(0).multi_processor_count, 160)
    each = tiles + ITEM_COST
    for b in range(1, blocks):
        u = n * heads * each * b // blocks
        at = u % each - ITEM_COST
        for x in range(max(at - 2, 0), min(at + 2, tiles)):
            marks[u // (heads * each), x] = True
    marks[::16, 0] = marks[8::16, tiles - 1] = True
    rng = np.random.default_rng(72)
    marks[rng.integers(0, n, 200), rng.integers(0, tiles, 200)] = True

    table = torch.from_numpy(marks.astype(np.int32)).cuda()
    desc = pkm.PagedCache(data=cache, page_table=table, layer_stride=0, page_stride=cache.stride(0),
                          kv_stride=cache.stride(1), slot_stride=cache.stride(2), num_layers=1, num_pages=2,
                          page_size=page, row_elems=heads * size,
                          cache_lengths=torch.full((n,), page * tiles - 1, dtype=torch.int32, device="cuda"))
    offsets = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(n, heads, device="cuda")
    ws = torch.empty(pkm.kv_attention_paged_workspace_size(n, heads, heads, size), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkm.kv_attention_paged(q, offsets, scale, desc, 0, out, ws, lse, status)
    assert status.item() == 0

    # the marked and the other page's keys, as often as they come
    k, v = (cache.double()[:, i].reshape(2 * page, heads, size) for i in range(2))
    count = torch.from_numpy(marks.sum(1)).cuda().double()
    times = torch.stack([tiles - count, count], 1).repeat_interleave(page, 1)[:, None]
    s = torch.einsum("nhc,thc->nht", q.double(), k) * scale
    w = s.exp() * times
    total = w.sum(-1)
    ref = torch.einsum("nht,thc->nhc", w, v) / total[..., None]
    spread = torch.einsum("nht,thc->nhc", w, v.abs()) / total[..., None]
    # as for short sums, scores off by e; and the running fp32 sums of weights (a tile at a time) and of
    # a stage's output (16 keys at a time, 2^15 times, at most 2^-23 each if the MMAs cut off)
    e = size * 2.0 ** -24 * (torch.einsum("nhc,thc->nht", q.double().abs(), k.abs()) * scale).amax(-1)
    long = 2.0 ** -8
    exact = total.log()
    off = (lse.double() - exact).abs()
    assert (off <= e + long + 2.0 ** -20 * (1 + exact.abs())).all(), (off.max(), off.argmax())
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12 + 2 * e[..., None] + 2 * long) * spread
    assert ((out.double() - ref).abs() <= tol).all()
    # and one tile more or less would have shown
    one = (total - w[..., page:].sum(-1) / count.clamp(min=1)[:, None]).log()
    marked = count > 0
    assert marked.sum() > blocks and (exact - one)[marked].min() > 10 * long
