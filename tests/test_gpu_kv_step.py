"""GPU: the calls on the paged K/V cache as a layer makes them -- projection into the cache
(kv_matmul_paged), rotary positions (kv_rope_paged), attention -- for chunks of prompts and then
token by token, alone and captured.  Each call is held to its definition on what the calls before it
left."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import dev
from kv_util import KvProblem, assert_kv_close
from spec_util import freqs_table, page_table
from test_gpu_kv_rope import assert_turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_mla_gb300  # noqa: F401


def bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


class Layer:
    """A layer's projections, cache and buffers for up to `rows` new tokens at a time."""
    K_IN, HEADS, KV_HEADS, SEQ, AXES, P = 256, 12, 2, 400, 3, 48

    def __init__(self, seed, batch, limit, rows, size, page, window, half):
        import paged_kv_mla_gb300 as pkm
        gen = np.random.default_rng(seed)
        torch.manual_seed(seed)
        self.pkm, self.size, self.page, self.window, self.half, self.batch = pkm, size, page, window, half, batch
        H, G, K = self.HEADS, self.KV_HEADS, self.K_IN
        self.w_q = torch.randn(K, H * size, device="cuda").bfloat16() * K ** -0.5
        self.w_kv = torch.randn(K, 2 * G * size, device="cuda").bfloat16() * K ** -0.5
        self.table, pages = page_table(gen, [limit] * batch, [0] * batch, page)
        self.cache = torch.zeros(2, pages, 2, page, G * size, dtype=torch.bfloat16, device="cuda")
        self.lengths = torch.zeros(batch, dtype=torch.int32, device="cuda")
        st = self.cache.stride()
        self.desc = pkm.PagedCache(data=self.cache, page_table=dev(self.table), layer_stride=st[0], page_stride=st[1],
                                   kv_stride=st[2], slot_stride=st[3], num_layers=2, num_pages=pages, page_size=page,
                                   row_elems=G * size, cache_lengths=self.lengths)
        self.freqs = torch.from_numpy(freqs_table(self.SEQ, self.P)).cuda()
        self.pair_axes = [j % self.AXES for j in range(self.P // 2)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.hidden = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
        self.positions = torch.zeros(self.AXES, rows, dtype=torch.int32, device="cuda")
        self.q = torch.zeros(rows, H, size, dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros_like(self.q)
        self.lse = torch.zeros(rows, H, device="cuda")
        n = pkm.kv_attention_paged_workspace_size(rows, H, G, size)
        self.workspace = torch.empty(n, dtype=torch.uint8, device="cuda")

    def attend(self, q, offsets, out, lse):
        if self.window:
            self.pkm.kv_window_attention_paged(q, offsets, self.size ** -0.5, *self.window, self.desc, 1, out,
                                               self.workspace, lse, self.status)
        else:
            self.pkm.kv_attention_paged(q, offsets, self.size ** -0.5, self.desc, 1, out, self.workspace, lse,
                                        self.status)

    def project(self, offsets, rows):
        self.pkm.kv_matmul_paged(self.hidden[:rows], offsets, self.w_kv, self.desc, 1, self.status)
        torch.matmul(self.hidden[:rows], self.w_q, out=self.q[:rows].view(rows, -1))

    def turn(self, offsets, rows):
        q = self.q[:rows]
        self.pkm.kv_rope_paged(offsets, self.positions[:, :rows].contiguous() if rows < len(self.q) else self.positions,
                               self.freqs, self.desc, 1, self.KV_HEADS, q=q, q_out=q, pair_axes=self.pair_axes,
                               half=self.half, dev_status=self.status)

    def problem(self, ctx, new):
        offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.uint32)
        window, sinks = self.window or (0, 0)
        return KvProblem(ctx, new, self.HEADS, self.KV_HEADS, self.size, self.page, self.size ** -0.5, window, sinks,
                         bits(self.q[:sum(new)]), bits(self.cache), self.table, offsets, 1)

    def step(self, ctx, new):
        """One step of all requests, every call checked; returns the problem of its attention."""
        rows = sum(new)
        self.hidden[:rows] = torch.randn(rows, self.K_IN, device="cuda").bfloat16()
        self.positions[:, :rows] = torch.randint(0, self.SEQ, (self.AXES, rows), device="cuda")
        self.lengths.copy_(torch.tensor(ctx))
        offsets = dev(np.concatenate([[0], np.cumsum(new)]).astype(np.uint32))
        self.project(offsets, rows)
        before, q = bits(self.cache), bits(self.q[:rows])
        self.turn(offsets, rows)
        factors = self.freqs.double().cpu().numpy().reshape(self.SEQ, -1, 2)
        at = self.positions[:, :rows].cpu().numpy()
        cs = factors[at[self.pair_axes].T, np.arange(self.P // 2)].reshape(rows, 1, self.P)
        p = self.problem(ctx, new)
        assert_turned(p.q, q, cs, self.P, self.half)
        r, rest = 0, p.cache.copy()
        for b, n in enumerate(new):
            t = ctx[b] + np.arange(n)
            place = (1, self.table[b, t // self.page], 0, t % self.page)
            shape = (n, self.KV_HEADS, self.size)
            if n:
                assert_turned(p.cache[place].reshape(shape), before[place].reshape(shape), cs[r:r + n], self.P, self.half)
            rest[place] = before[place]
            r += n
        assert np.array_equal(rest, before)
        self.attend(self.q[:rows], offsets, self.out[:rows], self.lse[:rows])
        assert self.status.item() == 0
        assert_kv_close(p, bits(self.out[:rows]), self.lse[:rows].cpu().numpy())
        return p


@pytest.mark.parametrize("size,page,window,half", [(128, 16, None, False), (64, 12, None, True),
                                                   (128, 32, (40, 3), True), (64, 8, (1, 1), False)])
def test_prompts_then_tokens(size, page, window, half):
    layer = Layer(size + page, 3, 260, 240, size, page, window, half)
    ctx = [0, 0, 0]
    for new in ([150, 1, 70], [0, 90, 33], [1, 1, 1], [1, 0, 1], [1, 1, 1]):
        p = layer.step(ctx, new)
        # the chunk's tokens one by one: each with the cache as long as it was for it
        for b in np.flatnonzero(np.asarray(new) > 1)[:1]:
            r0, n = int(p.offsets[b]), new[b]
            one = dev(np.array([0] * (b + 1) + [1] * (3 - b), np.uint32))
            out, lse = torch.empty_like(layer.out[:1]), torch.empty_like(layer.lse[:1])
            ref = p.reference()
            for i in (0, 1, n // 2, n - 1):
                layer.lengths[b] = ctx[b] + i
                layer.attend(layer.q[r0 + i:r0 + i + 1], one, out, lse)
                got = np.zeros_like(p.q)
                got[r0 + i] = bits(out[0])
                sums = np.zeros(p.q.shape[:2], np.float32)
                sums[r0 + i] = lse[0].cpu().numpy()
                assert_kv_close(p, got, sums, ref, rows=[r0 + i])
        ctx = [c + n for c, n in zip(ctx, new)]
    assert layer.status.item() == 0


def test_a_captured_step():
    """Four requests' single tokens, captured once and replayed while the requests grow: the bits of
    the calls made one by one."""
    layer = Layer(9, 4, 300, 300, 128, 16, (100, 2), True)
    ctx = [120, 0, 40, 100]
    layer.step([0, 0, 0, 0], ctx)
    offsets = torch.arange(5, dtype=torch.int32, device="cuda")
    rows = 4
    positions = torch.zeros(3, rows, dtype=torch.int32, device="cuda")

    def calls():
        layer.project(offsets, rows)
        layer.pkm.kv_rope_paged(offsets, positions, layer.freqs, layer.desc, 1, 2, q=layer.q[:rows],
                                q_out=layer.q[:rows], pair_axes=layer.pair_axes, half=True, dev_status=layer.status)
        layer.attend(layer.q[:rows], offsets, layer.out[:rows], layer.lse[:rows])

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        calls()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for i in range(4):
        layer.lengths.copy_(torch.tensor(ctx) + i)
        layer.hidden[:rows] = torch.randn(rows, layer.K_IN, device="cuda").bfloat16()
        positions.random_(0, layer.SEQ)
        kept = layer.cache.clone()
        calls()
        wanted = layer.out[:rows].clone(), layer.lse[:rows].clone(), layer.cache.clone()
        layer.cache.copy_(kept)
        layer.out.zero_()
        graph.replay()
        for got, want in zip((layer.out[:rows], layer.lse[:rows], layer.cache), wanted):
            assert torch.equal(got, want)
        p = layer.problem([c + i for c in ctx], [1] * 4)
        assert_kv_close(p, bits(layer.out[:rows]), layer.lse[:rows].cpu().numpy())
    assert layer.status.item() == 0
