"""Problems and 64-bit references for the speculative-decoding operators (tree attention,
query rotation, cache write at given positions, compaction).

Every cache element that no request owns is NaN (bf16) or the byte 0xFF (a quantised slot:
NaN codes, NaN rope values, NaN scales), so that a read of a stale slot shows."""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

from util import e4m3_decode_table

NAN_BF16 = 0x7FC0


def bf16_bits(x) -> np.ndarray:
    """float array -> bf16 bit patterns (round to nearest even)."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint16).copy()


def bf16_value(bits) -> np.ndarray:
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def page_table(gen, ctx, new, page, extra=2):
    """Shuffled pages for ctx + new tokens a request; unused entries point out of range."""
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    pages = sum(need) + extra
    order = gen.permutation(pages).astype(np.uint32)
    table = np.full((len(ctx), max(max(need, default=0), 1)), 0xFFFFFFF0, np.uint32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table, pages


def random_tree(gen, n):
    """Ancestor sets (Python integers, bit j = token j) of a random forest of n tokens."""
    bits = []
    for i in range(n):
        p = int(gen.integers(-1, i)) if i else -1
        bits.append((bits[p] if p >= 0 else 0) | (1 << i))
    return bits


def mask_array(rows_bits, words):
    out = np.zeros((len(rows_bits), words), np.uint32)
    for r, b in enumerate(rows_bits):
        for w in range(words):
            out[r, w] = (b >> (32 * w)) & 0xFFFFFFFF
    return out


@dataclass
class TreeProblem:
    ctx: list
    new: list
    heads: int
    rank: int
    rope: int
    page: int
    scale: float
    q: np.ndarray            # bf16 bits [rows, heads, C]
    cache: np.ndarray        # uint16 [layers, pages, page, slot] or uint8 slots
    table: np.ndarray
    offsets: np.ndarray
    mask: Optional[np.ndarray]
    layer: int
    quantised: bool

    @property
    def cols(self):
        return self.rank + self.rope

    @property
    def rows(self):
        return self.q.shape[0]

    def row_values(self, b):
        """fp64 latent rows [ctx + new, C] of request b."""
        t = np.arange(self.ctx[b] + self.new[b])
        cells = self.cache[self.layer, self.table[b][t // self.page], t % self.page]
        if not self.quantised:
            return bf16_value(cells[:, :self.cols])
        R, P = self.rank, self.rope
        codes = e4m3_decode_table()[cells[:, :R]]
        scale = np.ascontiguousarray(cells[:, R + 2 * P:R + 2 * P + R // 32]).view(np.float32)
        nope = codes.astype(np.float32) * np.repeat(scale, 128, 1)
        part = np.ascontiguousarray(cells[:, R:R + 2 * P]).view(np.uint16)
        return np.concatenate([bf16_value(bf16_bits(nope)), bf16_value(part)], 1)

    def seen(self, b):
        """bool [new, ctx + new]."""
        c, n = self.ctx[b], self.new[b]
        m = np.zeros((n, c + n), bool)
        m[:, :c] = True
        for i in range(n):
            for j in range(n):
                if self.mask is None:
                    m[i, c + j] = j <= i
                elif j < 32 * self.mask.shape[1]:
                    m[i, c + j] = (self.mask[self.offsets[b] + i, j // 32] >> np.uint32(j % 32)) & 1
        return m

    def reference(self):
        """(out, out_tol, lse, lse_tol) in fp64.

        Tolerances: bf16 output, half a step = 2^-8 |out|; every weight is rounded to bf16
        before the second product, 2^-8 relative, so 2^-8 sum w|v|; a score is a sum of C
        products in fp32 (error at most C 2^-24 sum |q k| times the scale, e below), which
        moves a weight by at most 2 e relative; 2^-12 covers the fp32 steps of the softmax."""
        H, R, C = self.heads, self.rank, self.cols
        out = np.zeros((self.rows, H, R))
        tol = np.zeros((self.rows, H, R))
        lse = np.full((self.rows, H), -np.inf)
        lse_tol = np.zeros((self.rows, H))
        for b in range(len(self.ctx)):
            n = self.new[b]
            if n == 0:
                continue
            keys = self.row_values(b)
            seen = self.seen(b)
            r0 = int(self.offsets[b])
            used = seen.any(0)
            keys = np.where(used[:, None], keys, 0.0)  # what nothing attends may be NaN
            for i in range(n):
                k = keys[seen[i]]
                if not len(k):
                    continue
                qi = bf16_value(self.q[r0 + i])
                s = qi @ k.T * self.scale
                e = C * 2.0 ** -24 * abs(self.scale) * (np.abs(qi) @ np.abs(k).T).max(1)
                m = s.max(1, keepdims=True)
                w = np.exp(s - m)
                l = w.sum(1)
                w /= l[:, None]
                v = k[:, :R]
                out[r0 + i] = w @ v
                size = w @ np.abs(v)
                tol[r0 + i] = (2.0 ** -8 * np.abs(out[r0 + i]) +
                               (2.0 ** -8 + 2.0 ** -12 + 2 * e)[:, None] * size)
                lse[r0 + i] = m[:, 0] + np.log(l)
                lse_tol[r0 + i] = e + 2.0 ** -20 * (1 + np.abs(lse[r0 + i]))
        return out, tol, lse, lse_tol


def quantised_slots(gen, shape, rank, rope, slot):
    x = gen.standard_normal((*shape, rank // 128, 128)).astype(np.float32)
    scale = (np.abs(x).max(-1) / np.float32(448)).astype(np.float32)
    codes = torch.from_numpy(x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    out = np.full((*shape, slot), 0xFF, np.uint8)
    out[..., :rank] = codes.reshape(*shape, rank)
    out[..., rank:rank + 2 * rope] = bf16_bits(gen.standard_normal((*shape, rope))).view(np.uint8)
    out[..., rank + 2 * rope:rank + 2 * rope + rank // 32] = scale.view(np.uint8)
    return out


def make_tree(seed, ctx, new, heads, rank=512, rope=64, page=16, tree=True, quantised=False,
              layers=2, layer=1, pad=0, scale=None, words=None, bits=None, q_std=1.0):
    gen = np.random.default_rng(seed)
    table, pages = page_table(gen, ctx, new, page)
    cols = rank + rope
    if quantised:
        payload = rank + 2 * rope + rank // 32
        slot = (payload + 15) // 16 * 16 + pad
        cache = np.full((layers, pages, page, slot), 0xFF, np.uint8)
    else:
        slot = cols + pad
        cache = np.full((layers, pages, page, slot), NAN_BF16, np.uint16)
    for b, (c, n) in enumerate(zip(ctx, new)):
        t = np.arange(c + n)
        if quantised:
            rows = quantised_slots(gen, (c + n,), rank, rope, slot)
            cache[layer, table[b][t // page], t % page] = rows
        else:
            cache[layer, table[b][t // page], t % page, :cols] = bf16_bits(
                gen.standard_normal((c + n, cols)))
    rows = sum(new)
    offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.uint32)
    mask = None
    if tree:
        words = words or max(1, -(-max(new) // 32))
        if bits is None:
            bits = [x for n in new for x in random_tree(gen, n)]
        mask = mask_array(bits, words)
    q = bf16_bits(gen.standard_normal((max(rows, 1), heads, cols)) * q_std)[:rows]
    return TreeProblem(list(ctx), list(new), heads, rank, rope, page,
                       scale if scale is not None else 1 / np.sqrt(128 + rope), q, cache, table,
                       offsets, mask, layer, quantised)


OUT_FILL, LSE_FILL = 0x7FA5, 12345.0


class DeviceTree:
    """A TreeProblem on the GPU, its outputs filled with sentinels."""

    def __init__(self, p: TreeProblem, extra_rows=0):
        import paged_kv_mla_gb300 as pkm
        from gpu_util import dev
        self.p = p
        self.q, self.cache, self.table = dev(p.q), dev(p.cache), dev(p.table)
        self.offsets = dev(p.offsets)
        self.lengths = dev(np.asarray(p.ctx, np.uint32))
        self.mask = None if p.mask is None else dev(p.mask)
        L, N, S, E = p.cache.shape
        sizes = dict(data=self.cache, page_table=self.table, layer_stride=N * S * E,
                     page_stride=S * E, slot_stride=E, num_layers=L, num_pages=N, page_size=S,
                     cache_lengths=self.lengths)
        if p.quantised:
            self.desc = pkm.QuantCache(kv_lora_rank=p.rank, rope_dim=p.rope, **sizes)
        else:
            self.desc = pkm.PagedCache(row_elems=p.cols, **sizes)
        rows = p.rows + extra_rows
        self.out = torch.full((rows, p.heads, p.rank), OUT_FILL, dtype=torch.int16, device="cuda")
        self.lse = torch.full((rows, p.heads), LSE_FILL, dtype=torch.float32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.workspace = self.new_workspace()

    def new_workspace(self):
        import paged_kv_mla_gb300 as pkm
        n = pkm.mla_tree_attention_paged_workspace_size(self.p.rows, self.p.heads, self.p.rank)
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self, stream=None, workspace=None, lse=True, out=None):
        import paged_kv_mla_gb300 as pkm
        p = self.p
        ws = self.workspace if workspace is None else workspace
        kw = dict(tree_mask=self.mask, lse=self.lse if lse else None, dev_status=self.status,
                  stream=stream)
        o = self.out if out is None else out
        if p.quantised:
            return pkm.mla_tree_attention_paged_qcache(self.q, self.offsets, p.scale, self.desc,
                                                       p.layer, o, ws, **kw)
        return pkm.mla_tree_attention_paged(self.q, self.offsets, p.scale, self.desc, p.layer,
                                            p.rank, p.rope, o, ws, **kw)

    def results(self):
        torch.cuda.synchronize()
        return (self.out.cpu().numpy().view(np.uint16), self.lse.cpu().numpy(),
                int(self.status.item()))


def assert_tree_close(p, out_bits, lse, ref=None):
    out, tol, ref_lse, lse_tol = ref or p.reference()
    got = bf16_value(out_bits[:p.rows])
    bad = ~(np.abs(got - out) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outputs outside tolerance; first at "
                           f"{tuple(np.argwhere(bad)[0])}: {got[bad][0]} for {out[bad][0]} "
                           f"+- {tol[bad][0]}")
    empty = np.isneginf(ref_lse)
    assert np.array_equal(empty, np.isneginf(lse[:p.rows]))
    if lse is not None and (~empty).any():
        d = np.abs(lse[:p.rows][~empty] - ref_lse[~empty])
        assert (d <= lse_tol[~empty]).all(), f"lse off by {d.max()} (allowed {lse_tol.max()})"


def rotate64(x, cs, half):
    """fp64 rotation of x [..., P] by (cos, sin) pairs cs [..., P]."""
    P = x.shape[-1]
    y = np.empty_like(x)
    for j in range(P // 2):
        i, k = (j, j + P // 2) if half else (2 * j, 2 * j + 1)
        y[..., i] = x[..., i] * cs[..., 2 * j] - x[..., k] * cs[..., 2 * j + 1]
        y[..., k] = x[..., i] * cs[..., 2 * j + 1] + x[..., k] * cs[..., 2 * j]
    return y


def freqs_table(positions, rope, base=10000.0):
    inv = base ** (-2 * np.arange(rope // 2) / rope)
    a = np.arange(positions)[:, None] * inv
    return np.stack([np.cos(a), np.sin(a)], -1).reshape(positions, rope).astype(np.float32)

