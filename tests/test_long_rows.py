"""The operators that read a long cache in part at their largest: a row of 2^20 positions, and
rows whose storage lies more than 2^31 elements into a layer."""
import numpy as np
import pytest

from select_ref import Rows
import test_evict
import test_sparse
import test_weights

pytestmark = pytest.mark.gpu


def test_a_row_of_a_million_keys():
    L = (1 << 20) - 9
    r = Rows(1, 1 << 20, 2, 1, 64, [L], seed=3)
    r.cache.enable_sparse(310)
    test_sparse.step(r, [1], 2, 300, 8)                 # 16382 candidate blocks
    test_weights.step(r, [1])                           # one pass: the scores fit
    test_weights.step(r, [3], 2)                        # a chunk: one more pass over K
    test_evict.evict(r, r, [0], [0], 5000, 64)          # weights past shared memory
    test_evict.check_state(r)
    assert r.cache.lens == [L + 5] and r.cache.slots == [5000]
    test_sparse.step(r, [1], 1, 3, 2)                   # positions at the rotary table's end
    test_weights.step(r, [1])
    assert r.cache.device_error() == 0


def test_rows_whose_scores_outgrow_their_room():
    """64 heads' scores of 330000 keys are more than a cache reserves room for: that row's
    weights take a pass of their own, beside a row and a chunk that go the usual ways."""
    r = Rows(3, 1 << 20, 64, 4, 64, [330000, 500, 70], seed=5)
    test_weights.step(r, [1, 1, 3])
    test_weights.step(r, [1, 0, 1], inplace=True)
    assert r.cache.device_error() == 0


@pytest.mark.parametrize("paged", [False, True])
def test_storage_past_two_to_the_31_elements(paged):
    """Dense: row 2's last heads lie at 3 x 8 x 2^20 x 128 elements; paged: the last head's
    blocks at as many."""
    M = 1 << 20
    r = Rows(3, M, 16, 8, 128, [70, 0, 400], seed=4, paged=paged, blocks=3 * M // 16 - 8)
    r.cache.enable_sparse(4)
    test_sparse.step(r, [1, 1], 1, 1, 1, rows=[0, 2])
    test_sparse.step(r, [40, 3], 1, 1, 1, rows=[2, 0], C=40)
    test_weights.step(r, [1, 1], rows=[0, 2])
    test_weights.step(r, [9, 2], rows=[2, 0], C=9)
    test_evict.evict(r, r, [2], [1], 130, 20)
    test_evict.evict(r, r, [2], [2], 200, 20)
    if not paged:                                       # (a paged view gathers every block)
        test_evict.check_state(r)
    test_sparse.step(r, [1, 1], 1, 1, 1, rows=[1, 2])
    test_weights.step(r, [1, 1], rows=[1, 2])
    assert r.cache.device_error() == 0
