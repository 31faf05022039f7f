"""GPU: what the two CTAs of a pair hand to each other (softmax weights, rows brought by loads,
drafts' values looked through) arrives whole: many runs over several tiles, with copies on
another stream taking bandwidth in different places, give the same bits, which are right."""
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


@pytest.mark.parametrize("page,quantised", [(128, False), (16, False), (12, False), (64, True)])
def test_same_bits_beside_copies(page, quantised):
    p = make_tree(760 + page, [900, 300, 1500], [5, 40, 1], 16, 512, 64, page=page,
                  quantised=quantised)
    g = DeviceTree(p)
    g.run()
    out, lse, status = g.results()
    assert status == 0
    assert_tree_close(p, out, lse)
    side = torch.cuda.Stream()
    a, b = (torch.zeros(32 << 20, dtype=torch.uint8, device="cuda") for _ in range(2))
    outs = [torch.zeros_like(g.out) for _ in range(30)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        with torch.cuda.stream(side):
            b[:(i + 1) << 20].copy_(a[:(i + 1) << 20])
        g.run(out=o)
    torch.cuda.synchronize()
    for o in outs:
        assert np.array_equal(o.cpu().numpy().view(np.uint16), out)
    assert g.status.item() == 0
