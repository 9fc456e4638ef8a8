"""Evictions that keep the last slots only (recent == keep), the plain sliding cut: no slot
competes, so every kept weight is one that the choice's CTA has only just read.  Rows of
several load passes (8192 slots each), held in shared memory and longer than that, into other
rows and in place; the moved accumulators are compared exactly."""
import numpy as np
import pytest

from select_ref import Rows
from test_evict import check_state, evict, kept_slots


@pytest.mark.gpu
@pytest.mark.parametrize("keep", [1, 700, 6000, 15000])
@pytest.mark.parametrize("alias", [False, True])
def test_held_rows_in_place(keep, alias):
    """keep = 15000 of 20000 slots: the accumulator's destination overlaps what is read."""
    r = Rows(4, 41000, 2, 2, 64, [20000, 9000, 40000, 16385], seed=keep)
    for _ in range(2):          # the second time every row keeps all of its slots
        evict(r, r, [0, 1, 2, 3], [0, 1, 2, 3], keep, keep, alias=alias)
    check_state(r)


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
def test_held_rows_into_another_cache(paged):
    kw = dict(kinds=(0, 1, 0), W=32, paged=paged)
    src = Rows(5, 30000, 4, 2, 64, [29000, 8192, 8193, 24576, 5], seed=1, **kw)
    dst = Rows(5, 30000, 4, 2, 64, [7, 0, 0, 900, 0], seed=2, **kw)
    for keep in (20000, 4096, 33):
        evict(src, dst, [0, 1, 2, 3, 4], [4, 2, 0, 1, 3], keep, keep)
        check_state(dst)


@pytest.mark.gpu
@pytest.mark.parametrize("alias", [False, True])
def test_rows_longer_than_shared_memory_holds(alias):
    r = Rows(2, 61000, 1, 1, 64, [60000, 52000], seed=3)
    evict(r, r, [0, 1], [0, 1], 45000, 45000, alias=alias)
    check_state(r)


def test_the_definition_keeps_the_last_slots():
    a = np.array([9, 8, 7, 1, 0], np.float32)
    assert kept_slots(a, 2, 2).tolist() == [3, 4]
    assert kept_slots(a, 5, 5).tolist() == [0, 1, 2, 3, 4]
