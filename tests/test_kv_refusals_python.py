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
