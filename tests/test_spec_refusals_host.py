"""Host memory is refused by the speculative-decoding entry points, whatever the state of CUDA in
the process, and the calls' other checks come before that."""
from __future__ import annotations

import threading

import pytest
import torch

import test_spec_refusals as r
from test_spec_refusals import INVALID, UNSUPPORTED, attention, b16, i32, paged, quant


@pytest.fixture(scope="module")
def pkm():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_mla_gb300
    return paged_kv_mla_gb300


@pytest.fixture(params=["as it is", "initialised"])
def state(request, pkm, monkeypatch):
    """CUDA as the process has it, and as after the first use of a device 0."""
    if request.param == "initialised":
        monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    return request.param


def calls(pkm):
    lat, g, f = b16(3, 576), torch.zeros(512), torch.zeros(8, 64)
    return {
        "attention": lambda: attention(pkm, paged(pkm)),
        "attention qcache": lambda: attention(pkm, quant(pkm)),
        "rope": lambda: r.rope(pkm, b16(3, 4, 16), b16(3, 4, 16)),
        "write": lambda: pkm.mla_cache_write_paged_at(lat, i32(3), i32(3), g, 1e-6, f, paged(pkm), 0,
                                                      512, 64, stream=0, check=False),
        "write qcache": lambda: pkm.mla_cache_write_paged_qcache_at(
            lat, i32(3), i32(3), g, 1e-6, f, quant(pkm), 0, stream=0, check=False),
        "compact": lambda: pkm.mla_cache_compact_paged(paged(pkm), 0, 1, i32(2, 3), i32(2), i32(2),
                                                       stream=0, check=False),
        "compact qcache": lambda: pkm.mla_cache_compact_paged_qcache(
            quant(pkm), 0, 1, i32(2, 3), i32(2), i32(2), stream=0, check=False)}


NAMES = ["attention", "attention qcache", "rope", "write", "write qcache", "compact", "compact qcache"]


@pytest.mark.parametrize("name", NAMES)
def test_host_memory_is_refused(pkm, state, name):
    assert calls(pkm)[name]() == INVALID


@pytest.mark.parametrize("name", NAMES)
def test_nothing_else_is_wrong_with_them(pkm, monkeypatch, name):
    """The control: but for the memory the calls would go on to the GPU."""
    monkeypatch.setattr(pkm, "_here", lambda device: True)
    pkm._lib.pkm_checks_only(1)
    try:
        assert calls(pkm)[name]() == pkm.PKM_ERR_CUDA
    finally:
        pkm._lib.pkm_checks_only(0)


def test_other_findings_come_first(pkm, state):
    """The refusals of test_spec_refusals.py hold in either state."""
    r.test_attention_alignment_and_null(pkm)
    r.test_nothing_to_do_is_fine(pkm)
    r.test_rope_arguments(pkm)
    r.test_compact_arguments(pkm)
    r.test_cache_write_at_needs_positions(pkm)
    r.test_views_that_the_calls_cannot_see(pkm)
    r.test_layers_too_long_for_loads(pkm)
    for rank, rope in [(32, 64), (576, 0), (520, 56), (512, 72), (64, 520)]:
        assert attention(pkm, paged(pkm, rank + rope), rank, rope) == UNSUPPORTED
    for rank, rope in [(64, 64), (640, 64), (512, 72), (128, 12)]:
        assert attention(pkm, quant(pkm, rank, rope), rank, rope) == UNSUPPORTED


def test_checks_alone_are_of_the_calling_thread(pkm):
    """A refusal under way in one thread does not stop another one's calls."""
    got = []

    def other():
        got.append(attention(pkm, paged(pkm, page_size=0)))
        pkm._lib.pkm_checks_only(0)

    pkm._lib.pkm_checks_only(1)
    t = threading.Thread(target=other)
    t.start()
    t.join()
    args = (b16(3, 4, 16), b16(3, 4, 16))
    x, y = args
    code = pkm._lib.mla_rope_heads(x.data_ptr(), 64, 16, i32(3).data_ptr(), 3, 4, 16,
                                   torch.zeros(4, 16).data_ptr(), 4, 0, y.data_ptr(), 64, 16, None, None)
    pkm._lib.pkm_checks_only(0)
    assert got == [INVALID] and code == pkm.PKM_ERR_CUDA
