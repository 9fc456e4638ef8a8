"""Calls captured into a CUDA graph that change what a cache's rows hold: an eviction replayed
once, and calls on paged rows whose new token opens a block."""
import numpy as np
import pytest

from select_ref import Rows, bits_of, dev
import test_evict
import test_sparse
import test_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_an_eviction(in_place, paged):
    import torch
    kw = dict(kinds=(0, 1, 0), W=40, paged=paged)
    lens = [1000, 300, 513, 90]
    src = Rows(4, 1100, 8, 2, 64, lens, seed=1, **kw)
    dst = src if in_place else Rows(4, 1100, 8, 2, 64, [20, 0, 700, 0], seed=2, **kw)
    warm = Rows(4, 1100, 8, 2, 64, lens, seed=1, **kw)              # kernels are loaded
    test_evict.evict(warm, warm, [0], [0], 100, 9)
    rows, to, keep, recent = [0, 1, 2, 3], [0, 1, 2, 3] if in_place else [2, 3, 0, 1], 200, 17
    acc = test_evict.accs(src, seed=5)
    acc_in = test_evict.to_dev(acc)
    acc_out = acc_in if in_place else [None if a is None else torch.full_like(a, -5.0)
                                       for a in acc_in]
    kept = [None if a is None else torch.full((4, 2, keep), -7, dtype=torch.int32, device="cuda")
            for a in acc_in]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dst.cache.evict_rows(src.cache, rows, to, keep, recent, acc_in, acc_out=acc_out,
                             kept=kept)
    g.replay()
    torch.cuda.synchronize()
    want = test_evict.expect(src, dst, rows, to, keep, recent, acc)
    for l in (0, 2):
        for i, (s, d) in enumerate(zip(rows, to)):
            m = want[l][i].shape[1]
            assert np.array_equal(kept[l].cpu().numpy()[i][:, :m], want[l][i])
            for h in range(2):
                assert np.array_equal(acc_out[l].cpu().numpy()[d, h, :m],
                                      acc[l][s, h][want[l][i][h]])
    test_evict.check_state(dst)
    if not in_place:
        test_evict.check_state(src)
    assert dst.cache.device_error() == 0


@pytest.mark.parametrize("call", ["sparse", "weights"])
@pytest.mark.parametrize("C", [1, 20])
def test_calls_that_open_a_block(call, C):
    import torch
    lens = [320, 48, 0]
    n_new = [1, C, 1]
    r = Rows(3, 500, 8, 2, 64, lens, seed=3, paged=True)
    r.cache.enable_sparse(4)
    if call == "weights":       # whatever a first call sets up
        test_weights.step(Rows(3, 500, 8, 2, 64, lens, seed=4, paged=True), n_new)
    q, k, v = r.tokens(3, C)
    qd, kd, vd = dev(q), dev(k), dev(v)
    out = torch.full((3, C, 8, 64), 12345.0, dtype=torch.bfloat16, device="cuda")
    sel = torch.full((3, C, 2, 4), -7, dtype=torch.int32, device="cuda")
    acc = torch.rand((3, 2, 500), device="cuda")
    before = acc.cpu().numpy()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        if call == "sparse":
            r.cache.append_sparse(0, qd, kd, vd, n_new, 1, sink=1, recent=2, out=out,
                                  selected=sel)
        else:
            r.cache.append_weights(0, qd, kd, vd, n_new, acc, acc, out=out)
    g.replay()
    torch.cuda.synchronize()
    if call == "sparse":
        test_sparse.check(r, 0, [0, 1, 2], n_new, q, k, v, 1, 1, 2, bits_of(out),
                          sel.cpu().numpy())
    else:
        test_weights.check(r, 0, [0, 1, 2], n_new, q, k, v, None, before, before, bits_of(out),
                           acc.cpu().numpy())
    r.cache.advance(n_new)
    for b, n in enumerate(n_new):
        r.K[0][b], r.V[0][b] = r.held(0, b, k[b, :n], v[b, :n], r.lens[b])
        r.lens[b] += n
    test_evict.check_state(r)
    test_sparse.step(r, [1, 1, 1], 1, 1, 2)
    assert r.cache.device_error() == 0


def test_a_sparse_call_made_twice_gives_the_same_bits():
    import torch
    r = Rows(5, 3000, 16, 4, 64, [2900, 20, 1333, 64, 700], seed=5)
    r.cache.enable_sparse(12)
    qkv = r.tokens(5, 40)
    n_new = [1, 40, 3, 0, 17]
    a = test_sparse.step(r, n_new, 1, 8, 2, qkv=qkv, advance=False)
    b = test_sparse.step(r, n_new, 1, 8, 2, qkv=qkv, advance=False)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
