"""The host side of the calls that read a long cache in part, run without a GPU on a stand-in
for the CUDA runtime (host_side.py): what they allocate, launch and count as known, and that a
call that fails has changed nothing."""
import pytest

import host_side
from host_side import Cache


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return host_side.build(str(tmp_path_factory.mktemp("host_side")))


def names(c):
    return [n for n, _ in c.launches()]


def test_the_stand_in_runs_a_step(lib):
    c = Cache(lib, kinds=(0, 1), W=8)
    assert c.rc == 0
    assert c.append([1, 40]) == 0 and c.append([1, 40], layer=1) == 0
    assert c.advance([1, 40]) == 0
    assert c.state()[0] == [1, 40]
    assert {"append_kernel", "decode_kernel", "state_kernel"} <= set(names(c))
    c.close()
    assert lib.fake_live_blocks() == 0


def test_bounds_of_a_failed_sparse_step_are_not_known(lib):
    """A single-token sparse step computes the bounds of its row's newest block in the launch of
    the selection; if that launch fails, the next call still has to compute them."""
    c = Cache(lib)
    c.fill([192, 65])
    assert lib.kv_sparse_enable(c.h, 4) == 0
    assert lib.kv_sparse_update(c.h, 0, host_side.i32([1]), 1, None) == 0
    assert c.sparse([1, 1], 1, 0, 2) == 0             # row 0: three blocks in a launch before
    assert c.advance([1, 1]) == 0
    assert c.append([63, 1]) == 0 and c.advance([63, 1]) == 0    # row 0: its fourth is complete
    assert lib.kv_sparse_update(c.h, 0, host_side.i32([1]), 1, None) == 0
    names(c)
    lib.fake_fail_launch(0)
    assert c.sparse([1, 1], 1, 0, 2) == 4             # KV_ERR_CUDA
    assert names(c) == []
    assert lib.kv_sparse_update(c.h, 0, None, 2, None) == 0
    assert names(c) == ["bounds_kernel"]
    assert lib.kv_sparse_update(c.h, 0, None, 2, None) == 0
    assert names(c) == []
    c.close()


def test_bounds_of_a_sparse_step_that_ran_are_known(lib):
    c = Cache(lib)
    c.fill([64, 127])
    assert lib.kv_sparse_enable(c.h, 4) == 0
    assert c.sparse([1, 1], 1, 0, 2) == 0             # bounds both rows' first blocks itself
    assert names(c)[-2:] == ["select_kernel", "decode_kernel"]
    assert lib.kv_sparse_update(c.h, 0, None, 2, None) == 0
    assert names(c) == []
    assert c.advance([1, 1]) == 0                     # row 1's second block is complete now
    assert lib.kv_sparse_update(c.h, 0, None, 2, None) == 0
    assert names(c) == ["bounds_kernel"]
    c.close()
