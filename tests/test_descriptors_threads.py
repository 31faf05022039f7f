"""Cache descriptors shared by threads: what one assigns holds for every later call, and no
thread changes a struct that another one's call reads."""
from __future__ import annotations

import sys
import threading

import pytest
import torch

from test_descriptors import make


@pytest.fixture(scope="module")
def pkm():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_mla_gb300
    return paged_kv_mla_gb300


@pytest.fixture()
def often():
    """Threads change places after every few instructions."""
    before = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    yield
    sys.setswitchinterval(before)


@pytest.mark.parametrize("quantised", [False, True])
def test_no_struct_outlives_an_assignment(pkm, often, quantised):
    c = make(pkm, quantised)
    stop = threading.Event()

    def calls():
        while not stop.is_set():
            c.c_struct()

    others = [threading.Thread(target=calls) for _ in range(2)]
    for t in others:
        t.start()
    stale = 0
    try:
        for size in range(1, 40001):
            c.page_size = size
            stale += c.c_struct().page_size != size
    finally:
        stop.set()
        for t in others:
            t.join()
    assert stale == 0


def _begun_before(pkm, c, assign):
    """The struct of another thread whose build read the fields and was then overtaken by
    `assign`, and that thread's next one."""
    read, go = threading.Event(), threading.Event()
    new_struct = type(c)._new_struct

    class Slow(type(c)):
        def _new_struct(self):
            s = new_struct(self)
            if threading.current_thread() is worker:
                read.set()
                go.wait(10)
            return s

    object.__setattr__(c, "__class__", Slow)
    got = []
    worker = threading.Thread(target=lambda: got.extend([c.c_struct(), c.c_struct()]))
    worker.start()
    assert read.wait(10)
    assign()
    go.set()
    worker.join()
    return got


@pytest.mark.parametrize("quantised", [False, True])
def test_a_build_that_an_assignment_overtakes_is_not_kept(pkm, quantised):
    c = make(pkm, quantised)

    def assign():
        c.page_size = 64

    first, second = _begun_before(pkm, c, assign)
    assert first.page_size in (2, 64) and second.page_size == 64
    assert c.c_struct().page_size == 64


@pytest.mark.parametrize("quantised", [False, True])
def test_threads_have_structs_of_their_own(pkm, quantised):
    c = make(pkm, quantised)
    mine, theirs = c.c_struct(), []
    t = threading.Thread(target=lambda: theirs.append(c.c_struct()))
    t.start()
    t.join()
    assert theirs[0] is not mine and c.c_struct() is mine
    old = mine.page_table, mine.max_pages_per_seq
    c.page_table = torch.zeros(2, 9, dtype=torch.int32)
    t = threading.Thread(target=lambda: theirs.append(c.c_struct()))
    t.start()
    t.join()
    assert (mine.page_table, mine.max_pages_per_seq) == old  # a call under way still reads it
    assert theirs[1].max_pages_per_seq == 9 == c.c_struct().max_pages_per_seq


@pytest.mark.parametrize("quantised", [False, True])
def test_table_and_its_width_are_of_one_tensor(pkm, quantised):
    """The table's address and width come from one reading of the field."""
    narrow, wide = (torch.zeros(2, n, dtype=torch.int32) for n in (4, 6))
    c = make(pkm, quantised)
    reads = []

    class Swapped(type(c)):
        def __getattribute__(self, name):
            if name == "page_table":
                reads.append(name)
                return narrow if len(reads) % 2 else wide
            return object.__getattribute__(self, name)

    object.__setattr__(c, "__class__", Swapped)
    for _ in range(4):
        s = c.c_struct()
        assert (s.page_table, s.max_pages_per_seq) in ((narrow.data_ptr(), 4), (wide.data_ptr(), 6))
