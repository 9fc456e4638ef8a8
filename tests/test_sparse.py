"""Sparse attention over selected blocks (kv_sparse_enable / update, kv_append_sparse).

The chosen blocks must equal the definition's exactly; the outputs are compared with a
64-bit attention over exactly those blocks, within a bound derived beside the reference
(select_ref.py).
"""
import ctypes

import numpy as np
import pytest

from select_ref import BLOCK, Rows, bits_of, check_out, choose, dev, f32, softmax_attend


def step(r, n_new, sink, top_k, recent, rows=None, C=None, layer=0, qkv=None, stream=None,
         advance=True, scale=1.0):
    """One sparse call on r's rows, checked against the reference; then the rows advance."""
    import torch
    rows = list(range(len(n_new))) if rows is None else rows
    C = C or max(1, max(n_new))
    q, k, v = qkv or r.tokens(len(rows), C, scale)
    per = sink + top_k + recent
    sel = torch.full((len(rows), C, r.Hk, per), -7, dtype=torch.int32, device="cuda")
    out = torch.full((len(rows), C, r.Hq, r.D), 12345.0, dtype=torch.bfloat16, device="cuda")
    r.cache.append_sparse(layer, dev(q), dev(k), dev(v), n_new, top_k, sink=sink, recent=recent,
                          rows=rows, out=out, selected=sel, stream=stream)
    torch.cuda.synchronize()
    got, chosen = bits_of(out), sel.cpu().numpy()
    check(r, layer, rows, n_new, q, k, v, sink, top_k, recent, got, chosen)
    if advance:
        r.cache.advance(n_new, rows)
        for i, (b, n) in enumerate(zip(rows, n_new)):
            r.K[layer][b], r.V[layer][b] = r.held(layer, b, k[i, :n], v[i, :n], r.lens[b])
            r.lens[b] += n
    return got, chosen


def check(r, layer, rows, n_new, q, k, v, sink, top_k, recent, got, chosen):
    for i, (b, n) in enumerate(zip(rows, n_new)):
        assert np.all(got[i, n:] == np.uint16(0x4641)), "padding written"
        assert np.all(chosen[i, n:] == -7), "padding's blocks written"
        if n == 0:
            continue
        L = r.lens[b]
        K, V = r.held(layer, b, k[i, :n], v[i, :n], L)
        qr = f32(r.rotated(q[i, :n], L)).reshape(n, r.Hk, r.rep, r.D)
        Kf, Vf = f32(K), f32(V).astype(np.float64)
        for t in range(n):
            slot = K.shape[1] - n + t      # L + t unless keys were evicted
            for g in range(r.Hk):
                want = choose(Kf[g], qr[t, g], slot, sink, top_k, recent)
                mine = chosen[i, t, g]
                assert mine[:len(want)].tolist() == want, f"row {b} token {t} head {g}"
                assert np.all(mine[len(want):] == -1)
                vis = np.zeros(slot + 1, bool)
                for blk in want:
                    vis[blk * BLOCK:(blk + 1) * BLOCK] = True
                _, ref, bound = softmax_attend(Kf[g, :slot + 1].astype(np.float64),
                                               Vf[g, :slot + 1], qr[t, g].astype(np.float64),
                                               vis)
                check_out(got[i, t, g * r.rep:(g + 1) * r.rep], ref, bound,
                          f"row {b} token {t} head {g}")


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("Hk,rep,D", [(2, 4, 64), (1, 16, 128), (2, 1, 128), (1, 9, 64),
                                      (3, 7, 128)])
def test_decode_lengths(Hk, rep, D, paged):
    lens = [0, 1, 62, 63, 64, 65, 127, 128, 700, 1023]
    r = Rows(len(lens), 1100, Hk * rep, Hk, D, lens, seed=D + rep, paged=paged)
    r.cache.enable_sparse(8)
    for _ in range(3):
        step(r, [1] * len(lens), 1, 3, 2)
    step(r, [1] * len(lens), 0, 5, 1)
    step(r, [1] * len(lens), 2, 0, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("sink,top_k,recent", [(0, 0, 1), (0, 1, 1), (3, 0, 1), (0, 31, 1),
                                               (1, 200, 7), (0, 1, 90)])
def test_counts(sink, top_k, recent):
    r = Rows(3, 6500, 8, 2, 64, [6400, 2111, 40], seed=5)
    r.cache.enable_sparse(sink + top_k + recent)
    step(r, [1, 1, 1], sink, top_k, recent)


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
def test_chunks_mixed_with_decodes(paged):
    lens = [0, 130, 61, 640, 300, 5]
    r = Rows(6, 1200, 8, 2, 64, lens, seed=11, paged=paged)
    r.cache.enable_sparse(6)
    step(r, [70, 1, 5, 33, 0, 64], 1, 2, 2, C=90)
    step(r, [1, 1, 130, 1, 2, 1], 1, 2, 1)
    step(r, [3, 0, 1], 0, 2, 2, rows=[5, 0, 3], C=3)


@pytest.mark.gpu
def test_more_queries_than_a_launch_holds():
    r = Rows(9, 500, 4, 2, 64, [0, 400, 3, 64, 200, 17, 0, 99, 1], seed=12)
    r.cache.enable_sparse(4)
    step(r, [64, 64, 64, 64, 64, 64, 64, 64, 64], 1, 1, 1)    # 576 queries


@pytest.mark.gpu
def test_more_queries_than_a_selection_holds():
    """1100 tokens, a row's chunk between two selections; 600 rows, of one or two tokens."""
    r = Rows(9, 700, 2, 1, 64, [0, 400, 3, 64, 200, 17, 0, 99, 1], seed=14)
    r.cache.enable_sparse(4)
    step(r, [130, 61, 130, 130, 130, 130, 130, 129, 130], 1, 1, 1)
    step(r, [1] * 9, 1, 2, 1)
    lens = [(37 * i) % 290 for i in range(600)]
    r = Rows(600, 300, 2, 1, 64, lens, seed=15)
    r.cache.enable_sparse(3)
    step(r, [1 + (i % 3 == 1) for i in range(600)], 0, 1, 1)
    step(r, [1] * 600, 1, 1, 1)


@pytest.mark.gpu
def test_far_apart_queries_of_one_call():
    """Token indices more than 2^16 apart in q."""
    import torch
    C = 40000
    r = Rows(4, C, 1, 1, 64, [100, 300, 20, 0], seed=13)
    r.cache.enable_sparse(3)
    n_new = [1, 2, 0, 1]
    q = np.zeros((4, C, 1, 64), np.uint16)
    k, v = q.copy(), q.copy()
    for x in (q, k, v):
        x[:, :2] = r.bits((4, 2, 1, 64))
    out = torch.full((4, C, 1, 64), 12345.0, dtype=torch.bfloat16, device="cuda")
    sel = torch.full((4, C, 1, 3), -7, dtype=torch.int32, device="cuda")
    r.cache.append_sparse(0, dev(q), dev(k), dev(v), n_new, 1, sink=1, recent=1, out=out,
                          selected=sel)
    torch.cuda.synchronize()
    check(r, 0, [0, 1, 2, 3], n_new, q, k, v, 1, 1, 1, bits_of(out), sel.cpu().numpy())


@pytest.mark.gpu
def test_ties_zeros_and_wide_values():
    """Equal blocks tie (the lowest win), zero keys and queries score 0, large and small
    magnitudes keep their order."""
    L = 64 * 9 + 10
    r = Rows(4, 700, 8, 2, 64, [L] * 4, seed=21)
    same = r.bits((2, 64, 64))
    r.K[0][0] = np.concatenate([same] * 10, 1)[:, :L]                  # all blocks alike
    r.K[0][1] = np.zeros((2, L, 64), np.uint16)                        # nothing to tell
    r.K[0][2] = (r.K[0][2] & 0x7FFF) | 0x0000                          # one sign
    scale = np.repeat(2.0 ** np.arange(-60, 70, 13), 64)[:L].astype(np.float32)
    r.K[0][3] = r.bits((2, L, 64))
    from select_ref import to_bits
    r.K[0][3] = to_bits(f32(r.K[0][3]) * scale[None, :, None] * np.float32(2.0 ** -57))
    for b in range(4):
        r.fill(b, L)
    r.cache.enable_sparse(6)
    q, k, v = r.tokens(4, 1)
    q[1, 0, :4] = 0
    k[1] = 0
    _, chosen = step(r, [1, 1, 1, 1], 1, 3, 2, qkv=(q, k, v))
    assert chosen[0, 0, 0].tolist() == [0, 1, 2, 3, 8, 9]
    assert chosen[1, 0, 0].tolist() == [0, 1, 2, 3, 8, 9]


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
def test_stale_slots_of_an_earlier_sequence(paged):
    """NaN and infinity left in a row's storage by an earlier sequence touch nothing."""
    L0 = 500
    bad = np.full((2, L0, 64), 0x7FC0, np.uint16)
    bad[:, ::3] = 0x7F80
    r = Rows(2, 600, 4, 2, 64, [L0, L0], seed=22, paged=paged, K=[[bad, bad]], V=[[bad, bad]])
    r.cache.enable_sparse(4)
    r.cache.update_sparse(0)
    r.cache.reset([0, 1])
    for b, L in enumerate([323, 7]):
        r.K[0][b], r.V[0][b] = r.bits((2, L, 64)), r.bits((2, L, 64))
        r.lens[b] = L
        r.fill(b, L)
    step(r, [1, 1], 1, 1, 1)
    step(r, [66, 1], 1, 1, 1)


@pytest.mark.gpu
def test_non_finite_keys_still_choose_valid_blocks():
    import torch
    L = 64 * 12 + 3
    r = Rows(1, 1000, 8, 2, 64, [L], seed=23)
    r.K[0][0][0, 130] = 0x7F80
    r.K[0][0][0, 300] = 0x7FC0
    r.K[0][0][1, 70] = 0xFF80
    r.fill(0, L)
    r.cache.enable_sparse(6)
    q, k, v = r.tokens(1, 1)
    q[0, 0, 5] = 0x7FC0
    q[0, 0, 6, 3] = 0x7F80
    sel = torch.full((1, 1, 2, 6), -7, dtype=torch.int32, device="cuda")
    r.cache.append_sparse(0, dev(q), dev(k), dev(v), [1], 3, sink=1, recent=2, selected=sel)
    for g in range(2):
        s = sel[0, 0, g].tolist()
        assert s == sorted(set(s)) and s[0] == 0 and s[-2:] == [11, 12]
    assert r.cache.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
def test_bounds_follow_every_way_a_row_changes(paged):
    """Dense appends, a repeated append of the same step, reset, copies, truncation, import."""
    import torch
    r = Rows(4, 900, 4, 2, 64, [300, 500, 64, 0], seed=31, paged=paged)
    r.cache.enable_sparse(4)
    args = (1, 1, 1)
    step(r, [1, 1, 1, 1], *args)
    # a dense append of several blocks
    q, k, v = r.tokens(4, 150)
    n = [150, 0, 70, 130]
    r.cache.append(0, dev(q), dev(k), dev(v), n)
    r.cache.advance(n)
    for b in range(4):
        r.K[0][b], r.V[0][b] = r.held(0, b, k[b, :n[b]], v[b, :n[b]], r.lens[b])
        r.lens[b] += n[b]
    step(r, [1, 1, 1, 1], *args)
    # the same step's tokens written twice: the second write counts
    step(r, [140, 64, 1, 70], *args, advance=False)
    step(r, [140, 64, 1, 70], *args)
    step(r, [1, 1, 1, 1], *args)
    # truncate row 0 in place, fork row 1 into row 2
    r.cache.copy_rows(r.cache, [0, 1], [0, 2], keep=[200, 300])
    r.K[0][0], r.V[0][0] = r.K[0][0][:, :200], r.V[0][0][:, :200]
    r.K[0][2], r.V[0][2] = r.K[0][1][:, :300], r.V[0][1][:, :300]
    r.lens[0], r.lens[2] = 200, 300
    step(r, [70, 1, 70, 1], *args)
    step(r, [1, 1, 1, 1], *args)
    # reset and refill with other keys, import over a row
    r.cache.reset([3])
    r.K[0][3] = r.V[0][3] = np.zeros((2, 0, 64), np.uint16)
    r.lens[3] = 0
    step(r, [1, 1, 1, 260], *args)
    r.K[0][1], r.V[0][1] = r.bits((2, 400, 64)), r.bits((2, 400, 64))
    r.lens[1] = 400
    r.fill(1, 400)
    r.cache.update_sparse(0, rows=[1, 3])
    step(r, [1, 1, 1, 1], *args)
    assert r.cache.device_error() == 0


@pytest.mark.gpu
def test_step_graph_between_sparse_steps():
    import torch
    r = Rows(2, 300, 4, 2, 64, [127, 190], seed=32)
    r.cache.enable_sparse(3)
    step(r, [1, 1], 0, 1, 1)
    q, k, v = r.tokens(2, 1)
    qd, kd, vd = dev(q), dev(k), dev(v)
    out = torch.empty_like(qd)
    g = r.cache.step_graph([qd], [kd], [vd], [out])
    g.launch()
    for b in range(2):
        r.K[0][b], r.V[0][b] = r.held(0, b, k[b], v[b], r.lens[b])
        r.lens[b] += 1
    step(r, [1, 1], 0, 1, 1)
    g.close()


@pytest.mark.gpu
def test_all_blocks_selected_is_dense_attention():
    """Every block selected: the dense call's outputs and the sparse one's are the same sums,
    but the dense kernel adds the step's own key after the others and the sparse one in its
    place, so each is held to the bound around the 64-bit value and not to the other's bits."""
    import torch
    lens = [1000, 63, 511]
    r = Rows(3, 1100, 16, 4, 128, lens, seed=41)
    r.cache.enable_sparse(20)
    q, k, v = r.tokens(3, 1)
    a = r.cache.append(0, dev(q), dev(k), dev(v), [1, 1, 1])
    sel = np.full((3, 1, 4, 20), -1)
    for i, L in enumerate(lens):
        sel[i, :, :, :L // 64 + 1] = np.arange(L // 64 + 1)
    check(r, 0, [0, 1, 2], [1, 1, 1], q, k, v, 5, 10, 5, bits_of(a), sel)
    step(r, [1, 1, 1], 5, 10, 5, qkv=(q, k, v))


@pytest.mark.gpu
def test_other_stream_and_a_captured_call():
    import torch
    r = Rows(2, 900, 8, 2, 64, [800, 333], seed=42)
    r.cache.enable_sparse(5)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(r, [1, 1], 1, 2, 2, stream=side)
    torch.cuda.synchronize()
    # capture one call without advancing; replays append and attend to new inputs
    q, k, v = r.tokens(2, 1)
    qd, kd, vd = dev(q), dev(k), dev(v)
    out = torch.full((2, 1, 8, 64), 12345.0, dtype=torch.bfloat16, device="cuda")
    sel = torch.full((2, 1, 2, 5), -7, dtype=torch.int32, device="cuda")
    args = (0, qd, kd, vd, [1, 1], 2)
    kw = dict(sink=1, recent=2, out=out, selected=sel)
    r.cache.append_sparse(*args, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.cache.append_sparse(*args, **kw)
    for _ in range(2):
        q, k, v = r.tokens(2, 1)
        qd.copy_(dev(q)), kd.copy_(dev(k)), vd.copy_(dev(v))
        g.replay()
        torch.cuda.synchronize()
        check(r, 0, [0, 1], [1, 1], q, k, v, 1, 2, 2, bits_of(out), sel.cpu().numpy())


@pytest.mark.gpu
@pytest.mark.parametrize("behind", [64, 400])
def test_a_captured_call_that_never_ran_leaves_no_bounds_behind(behind):
    """Bounds that a captured call would compute count only once they have been computed."""
    import torch
    r = Rows(2, 900, 8, 2, 64, [700, 128 + 63], seed=43)
    r.cache.enable_sparse(4)
    q, k, v = r.tokens(2, 1)
    qd, kd, vd = dev(q), dev(k), dev(v)
    # warm up on another cache, so that nothing is computed here before the capture
    w = Rows(2, 900, 8, 2, 64, [700, 128 + 63], seed=43)
    w.cache.enable_sparse(4)
    out = torch.empty_like(qd)
    w.cache.append_sparse(0, qd, kd, vd, [1, 1], 1, sink=0, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.cache.append_sparse(0, qd, kd, vd, [1, 1], 1, sink=0, out=out)
    if behind == 64:
        chunk = r.tokens(2, 2)
        step(r, [1, 1], 0, 1, 2, qkv=(q, k, v))
        step(r, [2, 2], 0, 1, 2, qkv=chunk)
    else:
        step(r, [70, 2], 0, 1, 2)
        step(r, [1, 1], 0, 1, 2)
    del g


@pytest.mark.gpu
def test_refusals_change_nothing():
    import torch
    import kv_cache_incremental_gb300 as kvi
    r = Rows(2, 200, 4, 2, 64, [100, 190], seed=51, kinds=(0, 1), W=8)
    q, k, v = (dev(x) for x in r.tokens(2, 1))
    with pytest.raises(kvi.KVError):
        r.cache.append_sparse(0, q, k, v, [1, 1], 1)              # not enabled
    with pytest.raises(kvi.KVError):
        r.cache.update_sparse(0)
    for m in (0, -1, 4097):
        with pytest.raises(kvi.KVError):
            r.cache.enable_sparse(m)
    r.cache.enable_sparse(4)
    with pytest.raises(kvi.KVError):
        r.cache.enable_sparse(4)                                  # once
    for kw in (dict(top_k=2), dict(top_k=-1), dict(top_k=1, sink=-1), dict(top_k=1, recent=0),
               dict(top_k=2**31 - 1, sink=0, recent=1)):
        with pytest.raises(kvi.KVError):
            r.cache.append_sparse(0, q, k, v, [1, 1], **kw)       # 1 + 2 + 2 > 4, signs
    with pytest.raises(kvi.KVError):
        r.cache.append_sparse(1, q, k, v, [1, 1], 1)              # a sliding layer
    with pytest.raises(kvi.KVError):
        r.cache.update_sparse(1)
    with pytest.raises(kvi.KVError):
        r.cache.update_sparse(0, rows=[0, 0])
    with pytest.raises(kvi.KVError):
        r.cache.append_sparse(0, q, k, v, [1, 2], 1)              # n_new > C
    with pytest.raises(TypeError):
        r.cache.append_sparse(0, q, k, v, [1, 1], 1,
                              selected=torch.zeros((2, 1, 2, 4), device="cuda"))
    with pytest.raises(ValueError):
        r.cache.append_sparse(0, q, k, v, [1, 1], 1, selected=torch.zeros(
            (2, 1, 2, 3), dtype=torch.int32, device="cuda"))
    big = [dev(x) for x in r.tokens(2, 20)]
    with pytest.raises(kvi.KVCacheFull):
        r.cache.append_sparse(0, *big, [1, 20], 1)
    assert r.cache.lens == [100, 190]
    h = kvi.KVCache(1, 64, 4, 2, 64, 8, [1])
    with pytest.raises(kvi.KVError):
        h.enable_sparse(4)                                        # no global layer


@pytest.mark.gpu
def test_pool_exhaustion_is_refused():
    import kv_cache_incremental_gb300 as kvi
    r = Rows(2, 128, 4, 2, 64, [48, 16], seed=52, paged=True, blocks=4)
    r.cache.enable_sparse(3)
    q, k, v = (dev(x) for x in r.tokens(2, 1))
    with pytest.raises(kvi.KVPoolExhausted):
        r.cache.append_sparse(0, q, k, v, [1, 1], 1, sink=0)
    assert r.cache.lens == [48, 16] and r.cache.free_blocks == 0


def test_null_and_range_checks_need_no_gpu():
    from kv_cache_incremental_gb300 import _lib
    lib = _lib.load()
    assert lib.kv_sparse_enable(None, 8) == 1
    assert lib.kv_sparse_update(None, 0, None, 0, None) == 1
    assert lib.kv_append_sparse(None, 0, None, None, None, 4, 1, None, None, 0, 1, 1, 1, None,
                                None, None) == 1


def test_reference_choice_on_a_worked_example():
    """Two-dimensional keys written out by hand: bounds, scores and the order of ties."""
    K = np.zeros((64 * 5, 2), np.float32)
    K[0:64] = [1, 0]
    K[64:128] = [0, 1]
    K[128:192] = [[-2, 1]] * 32 + [[1, 1]] * 32     # bounds [-2, 1] x [1, 1]
    K[192:256] = [0, 1]
    q = np.array([[1.0, 0.0]], np.float32)
    # scores: block 0 -> 127 levels of 1/127 = 1; block 1 -> 0; block 2 -> 1 (ceil 63.5 = 64
    # levels of 2/127, above 1); block 3 -> 0
    assert choose(K, q, 64 * 4 + 3, 0, 1, 1) == [2, 4]
    assert choose(K, q, 64 * 4 + 3, 0, 2, 1) == [0, 2, 4]
    assert choose(K, q, 64 * 4 + 3, 0, 3, 1) == [0, 1, 2, 4]
    q = np.array([[-1.0, 0.0]], np.float32)
    assert choose(K, q, 64 * 4 + 3, 1, 1, 1) == [0, 2, 4]
