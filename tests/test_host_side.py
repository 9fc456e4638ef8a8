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


def created_bytes(B, max_len, Hq, Hk, D, layers, sms=152):
    """Device memory of a dense cache of global layers, as kv_cache_create documents it."""
    kv = layers * 2 * B * Hk * (max_len + 1) * D * 2
    scratch = 2 * B * Hk * 64 * D * 2
    rope = max_len * (D // 2) * 8
    partials = (min(B, 512) * 32 * Hq + min(1024 * sms, B * Hq * 64 * 16)) * (D * 4 + 8)
    return kv + scratch + rope + partials + B * Hk * 4 + 16     # tickets, error word


@pytest.mark.parametrize("B,max_len,Hq,Hk,D,layers", [
    (16, 32768, 64, 8, 128, 6), (64, 8192, 32, 8, 128, 1), (1, 512, 8, 2, 64, 1),
    (3, 1 << 20, 64, 4, 64, 1)])
def test_memory_of_a_cache_that_counts_no_weights(lib, B, max_len, Hq, Hk, D, layers):
    """The memory of accumulated weights is allocated by a cache's first call that counts them,
    once, and by no other call."""
    c = Cache(lib, B, max_len, Hq, Hk, D, kinds=(0,) * layers)
    assert lib.fake_live_bytes() == created_bytes(B, max_len, Hq, Hk, D, layers)
    c.fill([min(300, max_len - 40)] * B)
    before = lib.fake_live_bytes()
    assert c.append([1] * B) == 0 and c.append([30] * B) == 0
    assert c.weights([0] * B) == 0 and lib.fake_live_bytes() == before
    assert c.weights([1] * B) == 0
    scores = min(B * Hq * (max_len + 3), 2 * 1024 * 152 * D)
    if scores <= min(1024 * 152, B * Hq * 64 * 16) * D:
        scores = 0                                     # the prefill partials hold them
    assert lib.fake_live_bytes() == before + B * 64 * Hq * 8 + 4 * scores
    after = lib.fake_live_bytes()
    assert c.weights([1] * B) == 0 and c.weights([30] * B, last=9) == 0
    assert lib.fake_live_bytes() == after
    c.close()
    assert lib.fake_live_blocks() == 0
    lib.fake_reset()


def test_a_first_counting_call_without_memory_changes_nothing(lib):
    for nth in range(2):                               # either of its two allocations
        c = Cache(lib, 2, 100000, 8, 2, 64, blocks=4000)
        c.fill([100, 50])
        was, held = c.state(), lib.fake_live_bytes()
        names(c)
        lib.fake_fail_malloc(nth)
        assert c.weights([1, 20]) == 5                 # KV_ERR_OOM
        assert names(c) == [] and c.state() == was and lib.fake_live_bytes() == held
        assert c.weights([1, 20]) == 0
        c.close()
        lib.fake_reset()


def test_a_first_counting_call_may_be_captured(lib):
    c = Cache(lib, 2, 30000, 8, 2, 64)
    c.fill([100, 50])
    lib.fake_capturing(1)
    assert c.weights([1, 20]) == 0
    assert lib.fake_bad_mallocs() == 0                 # none under a mode that refuses them
    lib.fake_reset()
    c.close()


def test_accumulators_that_overlap_in_part_are_refused(lib):
    c = Cache(lib)                                     # accumulators of 2 x 2 x 640 floats
    c.fill([100, 0])
    names(c)
    size = 2 * 2 * 640 * 4
    for d in (4, 640 * 4, size - 4):
        for a, b in ((0, d), (d, 0)):
            assert c.weights([1, 20], host_side.PTR + a, host_side.PTR + b) == 1
    assert names(c) == []
    assert c.weights([1, 20], host_side.PTR, host_side.PTR + size) == 0
    assert c.weights([1, 20], host_side.PTR + size, host_side.PTR) == 0
    assert c.weights([1, 20], host_side.PTR, host_side.PTR) == 0
    c.close()


def test_eviction_buffers_that_overlap_are_refused(lib):
    a = Cache(lib, kinds=(0, 1, 0), W=8)               # accumulators of 2 x 2 x 640 floats
    b = Cache(lib, kinds=(0, 1, 0), W=8)
    a.fill([300, 200])
    P, acc, kept = host_side.PTR, 2 * 2 * 640 * 4, 2 * 2 * 100 * 4
    was = a.state(), b.state()
    names(a)

    def call(dst, acc_in, acc_out, kept_):
        full = lambda x: None if x is None else [x[0], None, x[1]]
        return dst.evict([0, 1], a, [0, 1], 100, 9, full(acc_in), full(acc_out), full(kept_))

    A, B, C, D = (P + i * acc for i in range(4))       # next to one another
    K, L = P + 4 * acc, P + 4 * acc + kept
    for dst, args in (
            (b, ((A, B), (A, C), (K, L))),             # another cache: rows lie elsewhere
            (b, ((A, B), (C, B + 4), (K, L))),
            (a, ((A, B), (C, C), (K, L))),             # two layers written to one buffer
            (a, ((A, A), (A, C), (K, L))),             # one layer's weights read and written
            (a, ((A, B), (B, A), (K, L))),             # each layer's into the other's
            (a, ((A, B), (A + 4, C), (K, L))),         # in part
            (a, ((A, B), None, (K, K + 4))),           # kept lists
            (a, ((A, B), None, (K, B + acc - 4))),
            (a, ((A, B), (C, D), (K, D + acc - 4)))):
        assert call(dst, *args) == 1, args
    assert names(a) == [] and (a.state(), b.state()) == was
    for dst, args in ((b, ((A, B), (C, D), (K, L))), (a, ((A, B), (A, B), (K, L))),
                      (a, ((A, B), (C, D), (L, K))), (b, ((A, A), None, (K, L))),
                      (b, ((A, A + 8), (None, D), (K, L)))):
        assert call(dst, *args) == 0, args
    a.close()
    b.close()


@pytest.mark.parametrize("which", ["fake_fail_new", "fake_fail_malloc"])
def test_enabling_sparse_attention_without_memory_leaves_nothing_behind(lib, which):
    """Every allocation of the call, on the host or on the device, is the one that fails once."""
    nth = 0
    while True:
        c = Cache(lib, kinds=(0, 1, 0), W=8)
        held = lib.fake_live_bytes(), lib.fake_live_blocks()
        lib.fake_reset()
        getattr(lib, which)(nth)
        rc = lib.kv_sparse_enable(c.h, 4)
        lib.fake_reset()
        if rc == 0:
            assert nth >= 6                            # two layers' bounds, lists, tickets
            c.close()
            break
        assert rc == 5 and (lib.fake_live_bytes(), lib.fake_live_blocks()) == held, nth
        assert c.sparse([1, 1], 1) == 1                # still not enabled
        assert lib.kv_sparse_enable(c.h, 4) == 0
        c.close()
        assert lib.fake_live_blocks() == 0
        nth += 1


def evictions():
    """Paged rows 0 and 1 share blocks, row 2 has its own; (destination rows, source rows)."""
    return [([0, 2], [0, 2]), ([0, 2], [0, 1]), ([2, 1], [0, 1]), ([1], [2])]


@pytest.mark.parametrize("profile", [0, 1])
@pytest.mark.parametrize("dst,src", evictions())
def test_evictions_without_host_memory_change_nothing(lib, dst, src, profile):
    """Every host allocation of the call is the one that fails once."""
    P = host_side.PTR
    nth = 0
    while True:
        c = Cache(lib, B=3, kinds=(0, 1, 0), W=8, blocks=80)
        c.fill([300, 0, 130])
        assert lib.kv_copy_rows(c.h, host_side.i32([1]), c.h, host_side.i32([0]), None, 1,
                                None) == 0
        assert lib.kv_profile_enable(c.h, profile) == 0
        was = c.state()
        names(c)
        call = lambda: c.evict(dst, c, src, 100, 9, [P, None, P + (1 << 24)], None,
                               [P + (2 << 24), None, P + (3 << 24)])
        lib.fake_fail_new(nth)
        rc = call()
        lib.fake_fail_new(-1)
        if rc == 0:     # also when it is a launch's record that found no memory
            assert nth >= 10
            c.close()
            break
        assert rc == 5 and names(c) == [] and c.state() == was, nth
        assert call() == 0
        slots = c.state()[1]
        assert [slots[d] for d in dst] == [min(100, was[1][s]) for s in src]
        c.close()
        nth += 1
    lib.fake_reset()


def test_appends_that_run_out_of_host_memory_lose_no_block(lib):
    """A call that appends to paged rows and fails may have given them their blocks already
    (the call made again needs no others), but every block is free or some row's."""
    for call in (lambda c: c.sparse([1, 70, 1], 2), lambda c: c.weights([1, 70, 1], last=9)):
        nth = 0
        while True:
            c = Cache(lib, B=3, blocks=80)
            c.fill([304, 0, 128])                      # whole blocks: the next token needs one
            assert lib.kv_sparse_enable(c.h, 8) == 0
            lens = c.state()[0]
            lib.fake_fail_new(nth)
            rc = call(c)
            lib.fake_fail_new(-1)
            now, _, tables, free = c.state()
            assert free + sum(map(len, tables)) == 80 and now == lens, nth
            held = [b for t in tables for b in t]
            assert len(set(held)) == len(held)
            if rc != 0:
                assert rc == 5 and call(c) == 0
            c.close()
            nth += 1
            if rc == 0:
                break
    lib.fake_reset()
