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
