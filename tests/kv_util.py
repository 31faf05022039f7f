"""Problems and 64-bit references for the operators on the paged K/V cache (attention of new
tokens, with or without a window, and rotary positions with the cache write).

Every cache element that no request owns is NaN, so that a read of a stale slot shows."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

from spec_util import NAN_BF16, bf16_bits, bf16_value, page_table

OUT_FILL, LSE_FILL = 0x7FA5, 12345.0
# where the planes lie: [layer, page, plane, slot], [layer, plane, page, slot], [layer, page, slot, plane]
LAYOUTS = {"page": (0, 1, 2, 3), "plane": (0, 2, 1, 3), "slot": (0, 1, 3, 2)}


@dataclass
class KvProblem:
    ctx: list
    new: list
    heads: int
    kv_heads: int
    size: int
    page: int
    scale: float
    window: int              # 0: none
    sinks: int
    q: np.ndarray            # bf16 bits [rows, heads, D]
    cache: np.ndarray        # bf16 bits [layers, pages, planes, slots, row] by strides
    table: np.ndarray
    offsets: np.ndarray
    layer: int

    @property
    def rows(self):
        return self.q.shape[0]

    def plane(self, b, which):
        """fp64 rows [ctx + new, kv_heads, D] of request b."""
        t = np.arange(self.ctx[b] + self.new[b])
        pages = self.table[b, t // self.page]
        known = pages < self.cache.shape[1]  # given back: not to be read
        cells = self.cache[self.layer, np.where(known, pages, 0), which, t % self.page]
        out = bf16_value(cells[:, :self.kv_heads * self.size])
        out[~known] = np.nan
        return out.reshape(len(t), self.kv_heads, self.size)

    def seen(self, b):
        """bool [new, ctx + new]."""
        t = np.arange(self.ctx[b] + self.new[b])[None]
        p = self.ctx[b] + np.arange(self.new[b])[:, None]
        ok = t <= p
        if self.window:
            ok &= (t > p - self.window) | (t < self.sinks)
        return ok

    def reference(self):
        """(out, out_tol, lse, lse_tol) in fp64.

        Tolerances: bf16 output, half a step = 2^-8 |out|; every weight is rounded to bf16
        before the second product, 2^-8 relative, so 2^-8 sum w|v|; a score is a sum of D
        products in fp32 (error at most D 2^-24 sum |q k| times the scale, e below), which
        moves a weight by at most 2 e relative; 2^-12 covers the fp32 steps of the softmax."""
        H, D, group = self.heads, self.size, self.heads // self.kv_heads
        out = np.zeros((self.rows, H, D))
        tol = np.zeros((self.rows, H, D))
        lse = np.full((self.rows, H), -np.inf)
        lse_tol = np.zeros((self.rows, H))
        for b, n in enumerate(self.new):
            if n == 0:
                continue
            keys, values, seen = self.plane(b, 0), self.plane(b, 1), self.seen(b)
            r0 = int(self.offsets[b])
            for h in range(H):
                used = seen.any(0)
                k, v = keys[used, h // group], values[used, h // group]
                q = bf16_value(self.q[r0:r0 + n, h])
                ok = seen[:, used]
                clean_k, clean_v = np.nan_to_num(k, nan=0, posinf=0, neginf=0), np.where(np.isfinite(v), v, 0)
                s = np.where(ok, q @ clean_k.T * self.scale, -np.inf)
                e = D * 2.0 ** -24 * abs(self.scale) * np.where(ok, np.abs(q) @ np.abs(clean_k).T, 0).max(1)
                m = s.max(1, keepdims=True)
                w = np.exp(s - m)
                l = w.sum(1)
                w /= l[:, None]
                o = w @ clean_v
                bad = ~np.isfinite(v)
                if bad.any():  # a token that attends them has them in its sum
                    with np.errstate(invalid="ignore"):
                        for j in np.flatnonzero(bad.any(1)):
                            o[ok[:, j]] += np.where(bad[j], v[j], 0)
                out[r0:r0 + n, h] = o
                size = w @ np.abs(clean_v)
                tol[r0:r0 + n, h] = 2.0 ** -8 * np.abs(np.nan_to_num(o, posinf=0, neginf=0)) + \
                    (2.0 ** -8 + 2.0 ** -12 + 2 * e)[:, None] * size
                lse[r0:r0 + n, h] = m[:, 0] + np.log(l)
                lse_tol[r0:r0 + n, h] = e + 2.0 ** -20 * (1 + np.abs(lse[r0:r0 + n, h]))
        return out, tol, lse, lse_tol


def make_kv(seed, ctx, new, heads, kv_heads, size=128, page=16, window=0, sinks=0, layers=2,
            layer=1, layout="page", pad=0, scale=None, q_std=1.0):
    gen = np.random.default_rng(seed)
    table, pages = page_table(gen, ctx, new, page)
    row = kv_heads * size
    dims = (layers, pages, 2, page)
    order = LAYOUTS[layout]
    store = np.full([dims[i] for i in order] + [row + pad], NAN_BF16, np.uint16)
    cache = store.transpose(*[order.index(i) for i in range(4)], 4)
    for b, (c, n) in enumerate(zip(ctx, new)):
        t = np.arange(c + n)
        for plane in range(2):
            cache[layer, table[b][t // page], plane, t % page, :row] = bf16_bits(
                gen.standard_normal((c + n, row)))
    rows = sum(new)
    offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.uint32)
    q = bf16_bits(gen.standard_normal((max(rows, 1), heads, size)) * q_std)[:rows]
    return KvProblem(list(ctx), list(new), heads, kv_heads, size, page,
                     scale if scale is not None else size ** -0.5, window, sinks, q, cache, table,
                     offsets, layer)


def device_cache(cache, table, lengths, row):
    """PagedCache on the GPU of bf16 bits [layers, pages, planes, slots, row + pad] by strides, and
    its storage."""
    import paged_kv_mla_gb300 as pkm
    from gpu_util import dev
    base = cache
    while base.base is not None and base.base.dtype == cache.dtype:
        base = base.base
    data = dev(base)
    L, N, _, S, _ = cache.shape
    st = [x // 2 for x in cache.strides]
    desc = pkm.PagedCache(data=data, page_table=table, layer_stride=st[0], page_stride=st[1],
                          kv_stride=st[2], slot_stride=st[3], num_layers=L, num_pages=N, page_size=S,
                          row_elems=row, cache_lengths=lengths)
    return desc, torch.as_strided(data, cache.shape, st + [1] if len(st) == 4 else st)


class DeviceKv:
    """A KvProblem on the GPU, its outputs filled with sentinels."""

    def __init__(self, p: KvProblem, extra_rows=0, fused=False):
        from gpu_util import dev
        self.p = p
        self.q, self.table, self.offsets = dev(p.q), dev(p.table), dev(p.offsets)
        if fused:  # the queries among other columns of a wider row
            wide = torch.full((p.rows, p.heads + 3, p.size + 8), -1, dtype=torch.int16, device="cuda")
            wide[:, 1:p.heads + 1, :p.size] = self.q
            self.q = wide[:, 1:p.heads + 1, :p.size]
        self.lengths = dev(np.asarray(p.ctx, np.uint32))
        self.desc, self.cache = device_cache(p.cache, self.table, self.lengths, p.kv_heads * p.size)
        rows = p.rows + extra_rows
        self.out_all = torch.full((rows, p.heads, p.size), OUT_FILL, dtype=torch.int16, device="cuda")
        self.lse_all = torch.full((rows, p.heads), LSE_FILL, dtype=torch.float32, device="cuda")
        self.out, self.lse = self.out_all[:p.rows], self.lse_all[:p.rows]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.workspace = self.new_workspace()

    def new_workspace(self):
        import paged_kv_mla_gb300 as pkm
        n = pkm.kv_attention_paged_workspace_size(self.p.rows, self.p.heads, self.p.kv_heads, self.p.size)
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self, stream=None, workspace=None, lse=True, out=None):
        import paged_kv_mla_gb300 as pkm
        p = self.p
        ws = self.workspace if workspace is None else workspace
        o = self.out if out is None else out
        kw = dict(lse=self.lse if lse else None, dev_status=self.status, stream=stream)
        if p.window:
            return pkm.kv_window_attention_paged(self.q, self.offsets, p.scale, p.window, p.sinks,
                                                 self.desc, p.layer, o, ws, **kw)
        return pkm.kv_attention_paged(self.q, self.offsets, p.scale, self.desc, p.layer, o, ws, **kw)

    def results(self):
        torch.cuda.synchronize()
        return (self.out_all.cpu().numpy().view(np.uint16), self.lse_all.cpu().numpy(),
                int(self.status.item()))


def assert_kv_close(p, out_bits, lse, ref=None, rows=None):
    out, tol, ref_lse, lse_tol = ref or p.reference()
    pick = slice(None) if rows is None else rows
    got, out, tol = bf16_value(out_bits[:p.rows])[pick], out[pick], tol[pick]
    finite = np.isfinite(out)
    # not a number or an infinity: the same kind
    assert np.array_equal(np.isnan(got[~finite]), np.isnan(out[~finite]))
    inf = np.isinf(out)
    assert np.array_equal(got[inf], out[inf])
    bad = finite & ~(np.abs(got - np.where(finite, out, 0)) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outputs outside tolerance; first at "
                           f"{tuple(np.argwhere(bad)[0])}: {got[bad][0]} for {out[bad][0]} "
                           f"+- {tol[bad][0]}")
    if lse is not None:
        d = np.abs(lse[:p.rows][pick] - ref_lse[pick])
        assert (d <= lse_tol[pick]).all(), f"lse off by {d.max()} (allowed {lse_tol[pick].max()})"


def check(p, extra_rows=2, **kw):
    d = DeviceKv(p, extra_rows, **kw)
    d.run()
    out, lse, status = d.results()
    assert status == 0
    assert (out[p.rows:] == OUT_FILL).all() and (lse[p.rows:] == LSE_FILL).all()
    assert_kv_close(p, out, lse)
    return d
