"""The pieces of a row's keys that the chunk kernel joins itself (tickets in the cache) go in one
launch: were they in two and the second refused, the row's ticket would keep the first one's count
and the next call's join would come before its pieces.  Run without a GPU on a stand-in for the CUDA runtime
(host_side.py), and on a GPU against 64 bits."""
import pytest

import host_side
from host_side import PTR, Cache, i32


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return host_side.build(str(tmp_path_factory.mktemp("ticket_host")))


def chunk_grids(c):
    out = [c.lib.fake_launch_grid(i) for i in range(c.lib.fake_launches())
           if b"chunk_scored" in c.lib.fake_launch_name(i)]
    c.lib.fake_reset()
    return out


def call(c, what, n, layer=0):
    args = (c.h, layer, PTR, PTR, PTR, c.Hq, n, i32([n] * c.B), None, c.B)
    if what == "tree":
        return c.lib.kv_append_tree(*args, PTR, 0.0, None, PTR, None)
    return c.lib.kv_append_scored(*args, 5.0, None, None, None, PTR, None)


def rows(lib, B, keys):
    c = Cache(lib, B=B, max_len=keys + 100, Hq=8, Hk=1, D=64)
    c.fill([keys] * B)
    assert lib.kv_tree_enable(c.h) == 0
    c.lib.fake_reset()
    return c


@pytest.mark.parametrize("what", ["chunk", "tree"])
@pytest.mark.parametrize("B,keys,n", [(58, 60000, 4), (58, 200000, 17), (70, 200000, 17),
                                      (120, 60000, 4), (120, 60000, 17)])
def test_a_rows_pieces_share_a_launch(lib, B, keys, n, what):
    """Rows of one length have one number of pieces each, so every launch holds a multiple."""
    c = rows(lib, B, keys)
    assert call(c, what, n) == 0
    grids = chunk_grids(c)
    tiles = (8 * n + 127) // 128
    pieces = sum(grids) // (B * tiles)
    assert 1 < pieces <= 16 and sum(grids) == pieces * B * tiles
    assert len(grids) == -(-B // (512 // pieces))      # as few launches as that allows
    assert all(g % (pieces * tiles) == 0 for g in grids)
    c.close()


@pytest.mark.parametrize("what", ["chunk", "tree"])
def test_a_refused_launch_takes_whole_rows_with_it(lib, what):
    c = rows(lib, 120, 60000)
    assert call(c, what, 4) == 0
    whole = chunk_grids(c)
    assert len(whole) > 1
    pieces = sum(whole) // c.B
    for nth in range(len(whole)):
        lib.fake_fail_launch(1 + nth)                  # (the first launch stores the keys)
        assert call(c, what, 4) == 4                   # KV_ERR_CUDA
        assert all(g % pieces == 0 for g in chunk_grids(c))
        assert call(c, what, 4) == 0 and chunk_grids(c) == whole
    c.close()


@pytest.mark.gpu
def test_more_pieces_than_a_launch_holds():
    from scored_ref import parents_of
    from test_scored_long import Outputs
    lens = [20000 + 8 * b for b in range(120)]         # 600 pieces
    r = Outputs(120, 21000, 2, 1, 64, lens, seed=72)
    r.cache.enable_tree()
    r.call([2] * 120, cap=5.0, advance=False)
    n = [1 + b % 3 for b in range(120)]
    r.tree(n, [parents_of(r.rng, x, "tree") for x in n])
