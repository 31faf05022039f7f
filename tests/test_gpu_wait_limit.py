"""GPU: every form of the bounded wait gives up after its limit, not earlier and not much later,
and the kernels that use it run on as before."""
from __future__ import annotations

import time

import pytest
import torch

from spec_util import DeviceTree, assert_tree_close, make_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_mla_gb300  # noqa: F401


@pytest.mark.parametrize("ms", [1, 20, 300])
def test_waits_keep_their_limit(ms):
    import paged_kv_mla_gb300 as pkm
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    pkm.pkm_check_wait_timeout(st, ms)
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    assert int(st.item()) == pkm.PKM_ERR_TIMEOUT
    assert took >= ms * 1e-3
    p = make_tree(781, [300], [4], 4, page=16)
    g = DeviceTree(p)
    g.run()
    out, lse, status = g.results()
    assert status == 0
    assert_tree_close(p, out, lse)
