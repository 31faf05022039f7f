"""GPU: attention over the paged K/V cache with values that are not finite in many rows, where several
blocks share an item, in windows, and where weights underflow."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from kv_util import DeviceKv, check, make_kv
from spec_util import bf16_value

pytestmark = pytest.mark.gpu
INF, MINUS_INF, NAN = 0x7F80, 0xFF80, 0x7FC0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_mla_gb300  # noqa: F401


def put(p, b, t, values, cols=slice(None)):
    """Values of request b at positions t."""
    t = np.asarray(t)
    row = p.cache[p.layer, p.table[b, t // p.page], 1, t % p.page]
    row[:, :p.kv_heads * p.size][:, cols] = values
    p.cache[p.layer, p.table[b, t // p.page], 1, t % p.page] = row


@pytest.mark.parametrize("size", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(4, 1), (2, 2), (10, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3), (300, 130)])
def test_all_new_values(size, heads, kv_heads, window, sinks):
    """Every new value of one request is a NaN or an infinity, a column's sign by turns; the other
    requests', in the same items' blocks, are not."""
    p = make_kv(60, [500, 130, 90], [150, 333, 200], heads, kv_heads, size, 16, window, sinks, layers=1, layer=0)
    row = np.resize(np.array([NAN, INF, MINUS_INF, INF, INF], np.uint16), kv_heads * size)
    t = 130 + np.arange(333)
    put(p, 1, t, row)
    put(p, 1, t[40::50], row ^ 0x8000)  # both infinities in a column
    check(p)


@pytest.mark.parametrize("size", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (400, 3), (130, 200)])
@pytest.mark.parametrize("ctx,new", [(4000, 1), (3500, 40), (500, 200)])
def test_few_in_shared_items(size, window, sinks, ctx, new):
    p = make_kv(61, [ctx], [new], 4, 1, size, 16, window, sinks, layers=1, layer=0)
    last = ctx + new - 1
    for t, c, v in [(2, 0, INF), (129, 7, MINUS_INF), (ctx - 1, 9, NAN), (ctx - 1, 33, INF), (ctx, 33, INF),
                    (last, 40, MINUS_INF), (last - new // 2, 41, INF), (last, 42, NAN), (ctx, 50, INF),
                    (last, 50, MINUS_INF), (last - 399, 51, INF), (max(last - 129, 0), 52, MINUS_INF),
                    (ctx - 300, 53, NAN)]:
        put(p, 0, [t], v, c)
    check(p)


@pytest.mark.parametrize("size", [64, 128])
def test_short_items_that_take_turns(size):
    """Thousands of items of one tile, most of which need no look at their values, behind those that
    hold infinities."""
    gen = np.random.default_rng(62)
    new = gen.choice([1, 1, 1, 2, 3], 4000)
    ctx = np.where(new == 1, 127, 128 - new)
    p = make_kv(62, ctx.tolist(), new.tolist(), 2, 1, size, 128, layers=1, layer=0)
    for b in np.flatnonzero(new > 1)[::2]:
        put(p, b, [ctx[b] + new[b] - 1], INF, int(gen.integers(size)))
        put(p, b, [ctx[b]], MINUS_INF, int(gen.integers(size)))
    check(p)


@pytest.mark.parametrize("size", [64, 128])
@pytest.mark.parametrize("ctx,new", [(300, 1), (200, 180)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 2)])
def test_weights_that_underflow(size, ctx, new, window, sinks):
    """Attended infinities whose weights are often 0 in 32 bits: never a finite column; those that
    are not attended leave theirs as it is."""
    p = make_kv(63, [ctx], [new], 4, 1, size, 16, window, sinks, layers=1, layer=0, q_std=30.0)
    clean = p.reference()
    at = [1, ctx // 2, ctx, ctx + new - 1]
    for j, t in enumerate(at):
        put(p, 0, [t], INF, 3 + j)
    d = DeviceKv(p)
    d.run()
    out, lse, status = d.results()
    assert status == 0
    seen = p.seen(0)[:, at]  # [new, values]
    assert seen.any() and (new == 1 or not seen.all())
    got = bf16_value(out[:new])
    for j in range(len(at)):
        with_it = got[seen[:, j], :, 3 + j]
        assert (np.isnan(with_it) | (with_it == np.inf)).all()
        got[seen[:, j], :, 3 + j] = clean[0][seen[:, j], :, 3 + j]
    ref, tol = clean[:2]
    assert (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("size", [64, 128])
@pytest.mark.parametrize("ctx,new", [(20, 1), (3000, 1), (100, 60), (3000, 90)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 2)])
def test_scores_of_minus_infinity(size, ctx, new, window, sinks):
    """Keys whose scores are -inf weigh nothing; a row that attends no others is NaN, as 0 / 0 is, and
    its log-sum-exp -inf."""
    p = make_kv(65, [ctx, ctx], [new, new], 4, 2, size, 16, window, sinks, layers=1, layer=0)
    p.q[:, :2, 0] = 0x3F80  # 1, for the heads of the first head of keys
    t = np.arange(ctx + new)
    least = t % 3 == 1
    least[ctx:] = np.arange(new) % 2 == 1
    where = [np.flatnonzero(least), t]  # some keys of one request, all of the other
    for b in range(2):
        p.cache[0, p.table[b, where[b] // 16], 0, where[b] % 16, 0] = MINUS_INF
    d = DeviceKv(p)
    d.run()
    out, lse, status = d.results()
    assert status == 0
    assert np.isnan(bf16_value(out[new:2 * new, :2])).all() and (lse[new:2 * new, :2] == -np.inf).all()
    seen = p.seen
    p.seen = lambda b: seen(b) & ~least
    ref = p.reference()
    p.seen = seen
    rest = p.reference()
    some = seen(0) & ~least
    rows = np.flatnonzero(some.any(1))
    none = np.flatnonzero(~some.any(1))
    assert np.isnan(bf16_value(out[none, :2])).all() and (lse[none, :2] == -np.inf).all()
    for heads, (o, tol, l, l_tol), pick in ((slice(0, 2), ref, rows), (slice(2, 4), rest, np.arange(2 * new))):
        got = bf16_value(out[pick, heads])
        assert (np.abs(got - o[pick, heads]) <= tol[pick, heads]).all()
        assert (np.abs(lse[pick, heads] - l[pick, heads]) <= l_tol[pick, heads]).all()


def time_us(d):
    best = []
    for _ in range(8):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        d.run()
        b.record()
        torch.cuda.synchronize()
        best.append(a.elapsed_time(b) * 1e3)
    return min(best)


@pytest.mark.parametrize("size,window,sinks", [(128, 0, 0), (64, 512, 4)])
def test_a_request_that_is_not_finite_does_not_hold_up_others(size, window, sinks):
    """A diverged request's values cost a second look at its partly attended tiles (1.5 to 1.9 times
    the call), not one for every row, key and column."""
    p = make_kv(64, [2000, 1000], [512, 512], 32, 8, size, 128, window, sinks, layers=1, layer=0)
    clean = time_us(DeviceKv(p))
    put(p, 1, 1000 + np.arange(512), NAN)
    d = DeviceKv(p)
    took = time_us(d)
    out, _, status = d.results()
    assert status == 0
    assert np.isnan(bf16_value(out[512:1024])).all() and np.isfinite(bf16_value(out[:512])).all()
    assert took < 4 * clean, (took, clean)
