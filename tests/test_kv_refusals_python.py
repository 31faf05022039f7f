"""Arguments of the entry points on the paged K/V cache as Python gives them: whole numbers from arrays,
and numbers and tensors that the C calls would take for others."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from test_kv_refusals import GOES_ON, INVALID, attention, cache, lib, pkm, rope  # noqa: F401

AXES = [j % 3 for j in range(64)]


def named(x):
    return f"{type(x).__name__} {getattr(x, 'dtype', '')} {len(x) if hasattr(x, '__len__') else ''}"


@pytest.mark.parametrize("axes", [
    tuple(AXES), bytes(AXES), bytearray(AXES), np.array(AXES), np.array(AXES, np.int32), np.array(AXES, np.uint8),
    np.repeat(AXES, 2)[::2], torch.tensor(AXES), torch.tensor(AXES, dtype=torch.uint8)], ids=named)
def test_axes_of_pairs_in_any_array(pkm, axes, monkeypatch):
    seen = []
    run = pkm._run
    monkeypatch.setattr(pkm, "_run", lambda f, where, args, *rest: seen.append(args) or run(f, where, args, *rest))
    assert rope(pkm, cache(pkm), axes=3, pair_axes=AXES) == GOES_ON
    assert rope(pkm, cache(pkm), axes=3, pair_axes=axes) == GOES_ON
    given = [next(a for a in args if a.__class__ is bytes) for args in seen]
    assert len(given[0]) == 64 and given[0] == given[1]


@pytest.mark.parametrize("axes", [
    64, np.int64(64), np.array([0, 1] * 8, np.int32), np.array([0, 1] * 4), np.array(AXES, np.float32),
    torch.tensor(AXES, dtype=torch.float32), [0.0] * 64, np.array(AXES) + 256, np.array(AXES) - 1], ids=named)
def test_other_axes_are_refused(pkm, axes):
    assert rope(pkm, cache(pkm), axes=3, pair_axes=axes) == INVALID


@pytest.mark.parametrize("n", [2 ** 32, 2 ** 32 + 5, 2 ** 63, -2 ** 32 + 5, 2 ** 31])
def test_numbers_past_32_bits(pkm, n):
    """No cut-off: 2^32 + 5 is not a window of 5, nor 2^32 layer 0."""
    c = cache(pkm)
    assert attention(pkm, c, window=n) == INVALID and attention(pkm, c, window=7, sinks=n) == INVALID
    assert attention(pkm, c, layer=n) == INVALID and rope(pkm, c, layer=n) == INVALID
    assert attention(pkm, c, window=2 ** 31 - 1, sinks=2 ** 31 - 1) == GOES_ON
    assert attention(pkm, c, window=np.int64(7), sinks=np.int32(1), layer=np.int64(0)) == GOES_ON
    assert rope(pkm, c, layer=np.int64(0)) == GOES_ON


@pytest.mark.parametrize("scale,status", [(2.3e38, GOES_ON), (-2.3e38, GOES_ON), (2.4e38, INVALID), (-3.4e38, INVALID),
                                          (1e39, INVALID)])
def test_scales_whose_base_2_overflows(pkm, scale, status):
    """The scores' scale in base 2 would be infinite, and a score of 0 a NaN."""
    assert attention(pkm, cache(pkm), scale=scale) == status
    assert attention(pkm, cache(pkm), scale=scale, window=9) == status


@pytest.mark.parametrize("word,status", [
    (None, GOES_ON), (torch.zeros(1, dtype=torch.int32), GOES_ON), (torch.zeros(1, dtype=torch.int32).view(torch.uint32), GOES_ON),
    (torch.zeros((), dtype=torch.int32), GOES_ON), (torch.zeros(0, dtype=torch.int32), INVALID),
    (torch.zeros(1, dtype=torch.int64), INVALID), (torch.zeros(4, dtype=torch.uint8), INVALID)])
def test_the_status_word(pkm, word, status):
    c = cache(pkm)
    q, out, ws = torch.zeros(3, 8, 128, dtype=torch.int16), torch.zeros(3, 8, 128, dtype=torch.int16), workspace(pkm)
    rows = torch.zeros(3, dtype=torch.int32)
    kw = dict(dev_status=word, stream=0, check=False)
    assert pkm.kv_attention_paged(q, rows, 1.0, c, 0, out, ws, **kw) == status
    assert pkm.kv_window_attention_paged(q, rows, 1.0, 9, 1, c, 0, out, ws, **kw) == status
    assert pkm.kv_rope_paged(rows, rows, torch.zeros(16, 128), c, 0, 4, q=q, q_out=out, **kw) == status


def workspace(pkm):
    n = pkm.kv_attention_paged_workspace_size(3, 8, 4, 128)
    raw = torch.zeros(n + 256, dtype=torch.uint8)
    return raw[-raw.data_ptr() % 256:][:n]


@pytest.mark.gpu
def test_a_status_word_on_the_host():
    """Beside tensors on the GPU: refused, and nothing is launched that would write to it."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_mla_gb300 as m
    from kv_util import OUT_FILL, DeviceKv, make_kv
    d = DeviceKv(make_kv(70, [30], [5], 8, 2, 64, 16))
    d.status = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(m.PkmError):
        d.run()
    with pytest.raises(m.PkmError):
        m.kv_rope_paged(d.offsets, torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(1, 64, device="cuda"),
                        d.desc, d.p.layer, 2, q=d.q, q_out=d.out, dev_status=d.status)
    torch.cuda.synchronize()
    assert (d.out == OUT_FILL).all()
