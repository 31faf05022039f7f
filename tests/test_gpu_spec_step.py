"""GPU: the speculative-decoding operators as a serving step runs them: drafted trees written
into the cache at their depths, queries rotated and attended over the tree, the accepted path
compacted, and the next token attended -- against the same sequence without the rejected
drafts, written and attended token by token."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from spec_util import bf16_bits, bf16_value, freqs_table, mask_array, page_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_mla_gb300  # noqa: F401


def cu(a):
    a = np.ascontiguousarray(a)
    if a.dtype in (np.uint16, np.uint32):
        a = a.view(np.int16 if a.dtype == np.uint16 else np.int32)
    return torch.from_numpy(a).cuda()


class Server:
    """One cache, one layer, and the calls of a step."""

    def __init__(self, gen, ctx, room, heads, rank, rope, page, quantised):
        import paged_kv_mla_gb300 as pkm
        self.pkm, self.heads, self.rank, self.rope = pkm, heads, rank, rope
        self.quantised = quantised
        table, pages = page_table(gen, ctx, room, page)
        table[table >= pages] = 0
        self.table = cu(table)
        slot = (rank + 2 * rope + rank // 32 + 15) // 16 * 16 if quantised else rank + rope
        self.data = torch.full((1, pages, page, slot), -1,
                               dtype=torch.uint8 if quantised else torch.int16, device="cuda") \
            if not quantised else torch.full((1, pages, page, slot), 255, dtype=torch.uint8, device="cuda")
        self.lengths = torch.zeros(len(ctx), dtype=torch.int32, device="cuda")
        self.freqs = cu(freqs_table(400, rope))
        self.gamma = torch.ones(rank, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def cache(self):
        _, N, S, E = self.data.shape
        sizes = dict(data=self.data, page_table=self.table, layer_stride=N * S * E, page_stride=S * E,
                     slot_stride=E, num_layers=1, num_pages=N, page_size=S, cache_lengths=self.lengths)
        if self.quantised:
            return self.pkm.QuantCache(kv_lora_rank=self.rank, rope_dim=self.rope, **sizes)
        return self.pkm.PagedCache(row_elems=self.rank + self.rope, **sizes)

    def write(self, latent, offsets, positions):
        a = (cu(latent), cu(offsets), cu(positions), self.gamma, 1e-6, self.freqs, self.cache(), 0)
        if self.quantised:
            self.pkm.mla_cache_write_paged_qcache_at(*a, dev_status=self.status)
        else:
            self.pkm.mla_cache_write_paged_at(*a, self.rank, self.rope, dev_status=self.status)

    def attend(self, q, offsets, positions, mask=None):
        q, rows = cu(q), q.shape[0]
        self.pkm.mla_rope_heads(q[..., self.rank:], cu(positions), self.freqs, q[..., self.rank:],
                                dev_status=self.status)
        out = torch.zeros(rows, self.heads, self.rank, dtype=torch.int16, device="cuda")
        lse = torch.zeros(rows, self.heads, device="cuda")
        ws = torch.empty(self.pkm.mla_tree_attention_paged_workspace_size(rows, self.heads, self.rank),
                         dtype=torch.uint8, device="cuda")
        kw = dict(tree_mask=None if mask is None else cu(mask), lse=lse, dev_status=self.status)
        if self.quantised:
            self.pkm.mla_tree_attention_paged_qcache(q, cu(offsets), 0.1, self.cache(), 0, out, ws, **kw)
        else:
            self.pkm.mla_tree_attention_paged(q, cu(offsets), 0.1, self.cache(), 0, self.rank,
                                              self.rope, out, ws, **kw)
        assert self.status.item() == 0
        return bf16_value(out.cpu().numpy().view(np.uint16)), lse.cpu().numpy()

    def compact(self, accepted, counts):
        new = torch.zeros_like(self.lengths)
        f = self.pkm.mla_cache_compact_paged_qcache if self.quantised else self.pkm.mla_cache_compact_paged
        f(self.cache(), 0, 1, cu(accepted), cu(counts), new, dev_status=self.status)
        assert self.status.item() == 0
        self.lengths = new


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("heads,rank,rope,page", [(16, 512, 64, 64), (5, 128, 32, 12), (128, 256, 64, 16)])
def test_draft_verify_accept(heads, rank, rope, page, quantised):
    gen = np.random.default_rng(heads + page)
    ctx, C = [70, 3, 140], rank + rope
    trees = [[-1, 0, 0, 1, 2, 2, 5], [-1, 0], [-1, 0, 0, 0, 3, 1, 4, 4, 6]]
    paths = [[0, 2, 5, 6], [0], [0, 3, 4, 6, 8]]
    room = [len(t) + 4 for t in trees]
    offsets = np.cumsum([0] + [len(t) for t in trees]).astype(np.uint32)
    rows = int(offsets[-1])
    prompt = bf16_bits(gen.standard_normal((sum(ctx), C)))
    drafts = bf16_bits(gen.standard_normal((rows, C)))
    q = bf16_bits(gen.standard_normal((rows, heads, C)))
    last, q_last = bf16_bits(gen.standard_normal((3, C))), bf16_bits(gen.standard_normal((3, heads, C)))
    p_off = np.cumsum([0] + ctx).astype(np.uint32)
    p_pos = np.concatenate([np.arange(c) for c in ctx]).astype(np.uint32)
    bits, depth = [], []
    for t in trees:
        bb, dd = [], []
        for i, p in enumerate(t):
            bb.append((bb[p] if p >= 0 else 0) | 1 << i)
            dd.append(dd[p] + 1 if p >= 0 else 0)
        bits += bb
        depth.append(dd)
    pos = np.concatenate([np.add(c, d) for c, d in zip(ctx, depth)]).astype(np.uint32)

    tree = Server(gen, ctx, room, heads, rank, rope, page, quantised)
    tree.write(prompt, p_off, p_pos)
    tree.lengths = cu(np.array(ctx, np.uint32))
    tree.write(drafts, offsets, pos)
    out, lse = tree.attend(q, offsets, pos, mask_array(bits, 1))
    width = max(len(p) for p in paths)
    acc = np.array([p + [0] * (width - len(p)) for p in paths], np.uint32)
    tree.compact(acc, np.array([len(p) for p in paths], np.uint32))
    assert tree.lengths.tolist() == [c + len(p) for c, p in zip(ctx, paths)]
    one = np.arange(4, dtype=np.uint32)
    end = np.array([c + len(p) for c, p in zip(ctx, paths)], np.uint32)
    tree.write(last, one, end)
    out_last, lse_last = tree.attend(q_last, one, end)

    # the accepted tokens alone, one step at a time
    flat = Server(gen, ctx, room, heads, rank, rope, page, quantised)
    flat.write(prompt, p_off, p_pos)
    flat.lengths = cu(np.array(ctx, np.uint32))
    for step in range(width):
        live = [b for b in range(3) if step < len(paths[b])]
        pick = [int(offsets[b]) + paths[b][step] for b in live]
        off = np.cumsum([0] + [1 if b in live else 0 for b in range(3)]).astype(np.uint32)
        at = np.array([ctx[b] + step for b in live], np.uint32)
        flat.write(drafts[pick], off, at)
        o, l = flat.attend(q[pick], off, at)
        # the same keys in another order of addition: twice the rounding of the weights and
        # of the result, 2 (2^-8 |out| + 2^-8 sum w|v|), with |v| < 6 for these rows
        assert np.abs(o - out[pick]).max() <= 2 * 2.0 ** -8 * (np.abs(o).max() + 6.0)
        assert np.abs(l - lse[pick]).max() <= 1e-4
        flat.lengths += cu(np.array([1 if b in live else 0 for b in range(3)], np.int32))
    assert flat.lengths.tolist() == tree.lengths.tolist()
    flat.write(last, one, end)
    o, l = flat.attend(q_last, one, end)
    # the caches hold the same rows at the same positions: the same bits
    assert np.array_equal(o, out_last) and np.array_equal(l, lse_last)
