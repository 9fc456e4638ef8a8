"""What ends a row's drafts, on a stand-in for the CUDA runtime (host_side.py): a replayed decode step as
well.  And the refusals on caches with hybrid layers."""
import ctypes

import pytest

import host_side
import kv_cache_incremental_gb300 as kvi
from host_side import PTR, Cache, i32


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return host_side.build(str(tmp_path_factory.mktemp("drafts_host")))


def draft(c, n_new):
    for layer in range(len(c.kinds)):
        assert c.lib.kv_append_tree(c.h, layer, PTR, PTR, PTR, c.Hq, max(n_new), i32(n_new), None,
                                    len(n_new), PTR, 0.0, None, PTR, None) == 0


def accept(c, tokens):
    """Token 0 of each row that is in `tokens`."""
    n = [int(b in tokens) for b in range(c.B)]
    return c.lib.kv_accept_tree(c.h, i32([0] * c.B), 1, i32(n), None, c.B, None)


def step_graph(c, rows):
    g = ctypes.c_void_p()
    bufs = (ctypes.c_void_p * len(c.kinds))(*[PTR] * len(c.kinds))
    assert c.lib.kv_step_graph_create(c.h, ctypes.byref(g), bufs, bufs, bufs, bufs, c.Hq,
                                      i32(rows), len(rows)) == 0
    return g


@pytest.mark.parametrize("blocks", [None, 200])
def test_a_replayed_step_ends_its_rows_drafts(lib, blocks):
    c = Cache(lib, B=3, kinds=(0, 1), W=8, blocks=blocks)
    c.fill([40, 50, 30])
    assert lib.kv_tree_enable(c.h) == 0
    g = step_graph(c, [0, 2])                          # before the drafts, replayed after them
    draft(c, [5, 5, 5])
    assert accept(c, [0, 1, 2]) == 0                   # (a path does not end them, its advance does)
    assert lib.kv_step_graph_launch(g, None) == 0
    assert c.state()[0] == [41, 50, 31]
    was = c.state()
    assert accept(c, [0]) == 1 and accept(c, [2]) == 1 and accept(c, [0, 1, 2]) == 1
    assert c.state() == was
    assert accept(c, [1]) == 0                         # a row that is not in the graph
    draft(c, [5, 5, 5])
    assert accept(c, [0, 1, 2]) == 0
    lib.kv_step_graph_destroy(g)
    c.close()
    assert lib.fake_live_blocks() == 0


def test_a_row_that_does_not_advance_keeps_its_drafts(lib):
    c = Cache(lib, B=2)
    c.fill([40, 50])
    assert lib.kv_tree_enable(c.h) == 0
    draft(c, [5, 5])
    assert c.advance([0, 1]) == 0
    assert accept(c, [1]) == 1 and accept(c, [0]) == 0
    c.close()


@pytest.mark.parametrize("kinds", [[kvi.KV_HYBRID_FULL, kvi.KV_HYBRID_LOCAL],
                                   [kvi.KV_GLOBAL, kvi.KV_HYBRID_FULL]])
def test_hybrid_layers_are_refused(lib, kinds):
    c = Cache(lib, B=2, max_len=64, kinds=kinds, W=8)
    assert c.rc == 0
    assert lib.kv_tree_enable(c.h) == 1
    one = i32([1, 1])
    for layer, kind in enumerate(kinds):
        rc = 0 if kind == kvi.KV_GLOBAL else 1
        lib.fake_reset()
        assert lib.kv_store(c.h, layer, PTR, PTR, 1, one, None, 2, None) == rc
        assert lib.kv_append_scored(c.h, layer, PTR, PTR, PTR, c.Hq, 1, one, None, 2, 1.0, None,
                                    None, None, PTR, None) == rc
        assert lib.kv_append_tree(c.h, layer, PTR, PTR, PTR, c.Hq, 1, one, None, 2, PTR, 1.0, None,
                                  PTR, None) == 1
        assert bool(lib.fake_launches()) == (rc == 0)
    c.close()
