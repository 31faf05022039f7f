"""GPU: more requests than the attention's threads, each of which then counts several."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from spec_util import DeviceTree, assert_tree_close, make_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_mla_gb300  # noqa: F401


@pytest.mark.parametrize("requests", [640, 641, 1300, 2000])
@pytest.mark.parametrize("page,quantised", [(16, False), (12, False), (32, True)])
def test_more_requests_than_threads(requests, page, quantised):
    gen = np.random.default_rng(requests + page)
    ctx = gen.integers(0, 40, requests).tolist()
    new = gen.choice([0, 0, 1, 1, 2, 5], requests).tolist()
    ctx[3], ctx[requests - 2], new[requests - 2], new[0] = 700, 300, 9, 0
    p = make_tree(800 + requests, ctx, new, 3, 128, 16, page=page, quantised=quantised)
    g = DeviceTree(p)
    g.run()
    out, lse, status = g.results()
    assert status == 0
    assert_tree_close(p, out, lse)
