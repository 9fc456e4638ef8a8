"""Accumulated attention weights (kv_append_weights): every key's weight, and the attention
outputs beside it, against a 64-bit softmax within bounds derived in select_ref.py."""
import numpy as np
import pytest

from select_ref import Rows, bits_of, check_out, dev, f32, softmax_attend, weight_error


def step(r, n_new, last=None, rows=None, C=None, layer=0, inplace=False, advance=True,
         stream=None, qkv=None):
    import torch
    rows = list(range(len(n_new))) if rows is None else rows
    C = C or max(1, max(n_new))
    q, k, v = qkv or r.tokens(len(rows), C)
    shape = (r.B, r.Hk, r.max_len)
    before = r.rng.random(shape, dtype=np.float32) * np.float32(5)
    slots = r.cache.slots
    for b in range(r.B):
        before[b, :, slots[b]:] = np.nan        # not yet keys: must not be read
    acc_in = torch.from_numpy(before.copy()).cuda()
    acc_out = acc_in if inplace else torch.full(shape, -3.0, device="cuda")
    untouched = acc_out.cpu().numpy()
    out = torch.full((len(rows), C, r.Hq, r.D), 12345.0, dtype=torch.bfloat16, device="cuda")
    r.cache.append_weights(layer, dev(q), dev(k), dev(v), n_new, acc_in, acc_out, last=last,
                           rows=rows, out=out, stream=stream)
    torch.cuda.synchronize()
    got, acc = bits_of(out), acc_out.cpu().numpy()
    check(r, layer, rows, n_new, q, k, v, last, before, untouched, got, acc)
    if advance:
        r.cache.advance(n_new, rows)
        for i, (b, n) in enumerate(zip(rows, n_new)):
            r.K[layer][b], r.V[layer][b] = r.held(layer, b, k[i, :n], v[i, :n], r.lens[b])
            r.lens[b] += n
    return got, acc


def check(r, layer, rows, n_new, q, k, v, last, before, untouched, got, acc):
    seen = set()
    for i, (b, n) in enumerate(zip(rows, n_new)):
        assert np.all(got[i, n:] == np.uint16(0x4641)), "padding written"
        if n == 0:
            continue
        seen.add(b)
        L = r.lens[b]
        K, V = r.held(layer, b, k[i, :n], v[i, :n], L)
        s0 = K.shape[1] - n
        qr = f32(r.rotated(q[i, :n], L)).reshape(n, r.Hk, r.rep, r.D).astype(np.float64)
        Kf, Vf = f32(K).astype(np.float64), f32(V).astype(np.float64)
        counted = n if last is None else min(n, last)
        for g in range(r.Hk):
            want = np.zeros(s0 + n)
            want[:s0] = before[b, g, :s0]
            slack = np.abs(want) * 2.0 ** -24
            for t in range(n):
                m = s0 + t + 1
                w, ref, bound = softmax_attend(Kf[g, :m], Vf[g, :m], qr[t, g], np.ones(m, bool))
                check_out(got[i, t, g * r.rep:(g + 1) * r.rep], ref, bound,
                          f"row {b} token {t} head {g}")
                if t >= n - counted:
                    want[:m] += w.sum(0)
                    slack[:m] += (w * weight_error(qr[t, g], Kf[g, :m])[:, None]).sum(0)
            # float32 sums of counted * rep weights in any order
            slack += want * (counted * r.rep + 2) * 2.0 ** -24 + 1e-37
            err = np.abs(acc[b, g, :s0 + n].astype(np.float64) - want)
            assert np.all(err <= slack), (b, g, int(np.argmax(err - slack)), (err / slack).max())
            rest, was = acc[b, g, s0 + n:], untouched[b, g, s0 + n:]
            assert np.array_equal(rest, was, equal_nan=True), "slots past the row written"
    for b in set(range(r.B)) - seen:
        assert np.array_equal(acc[b], untouched[b], equal_nan=True), "another row written"


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("Hk,rep,D", [(2, 4, 64), (1, 16, 128), (2, 1, 128), (1, 9, 64),
                                      (3, 7, 128), (1, 8, 64)])
def test_decode_lengths(Hk, rep, D, paged):
    lens = [0, 1, 15, 16, 63, 64, 127, 128, 700, 1500]
    r = Rows(len(lens), 1600, Hk * rep, Hk, D, lens, seed=D + rep, paged=paged)
    step(r, [1] * len(lens))
    step(r, [1] * len(lens), inplace=True)


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("last", [None, 1, 7, 32])
def test_chunks(last, paged):
    lens = [0, 130, 61, 640, 300, 5]
    r = Rows(6, 1200, 8, 2, 64, lens, seed=11, paged=paged)
    step(r, [70, 1, 5, 33, 0, 64], last, C=90)
    step(r, [1, 1, 130, 1, 2, 1], last, inplace=True)
    step(r, [3, 0, 1], last, rows=[5, 0, 3], C=3)


@pytest.mark.gpu
@pytest.mark.parametrize("Hk,rep,D", [(1, 16, 128), (3, 3, 128), (2, 1, 64)])
def test_chunk_shapes(Hk, rep, D):
    r = Rows(3, 700, Hk * rep, Hk, D, [0, 333, 129], seed=12)
    step(r, [66, 40, 2])
    step(r, [1, 9, 30], 5)


@pytest.mark.gpu
def test_more_rows_than_a_launch_holds():
    B = 520
    lens = [(7 * b) % 90 for b in range(B)]
    r = Rows(B, 100, 2, 1, 64, lens, seed=13)
    step(r, [1 + (b % 3) for b in range(B)], C=3)


@pytest.mark.gpu
def test_long_row_in_many_splits():
    r = Rows(1, 40000, 4, 1, 128, [39000], seed=14)
    step(r, [1])
    step(r, [5], 2)


@pytest.mark.gpu
def test_stale_nan_slots_touch_nothing():
    L0 = 500
    bad = np.full((2, L0, 64), 0x7FC0, np.uint16)
    r = Rows(2, 600, 4, 2, 64, [L0, L0], seed=22, K=[[bad, bad]], V=[[bad, bad]])
    r.cache.reset([0, 1])
    for b, L in enumerate([323, 7]):
        r.K[0][b], r.V[0][b] = r.bits((2, L, 64)), r.bits((2, L, 64))
        r.lens[b] = L
        r.fill(b, L)
    step(r, [1, 1])
    step(r, [66, 3])


@pytest.mark.gpu
def test_large_scores():
    """Scores of several hundred: the weights of a softmax that is nearly one key."""
    r = Rows(2, 400, 8, 2, 64, [300, 130], seed=23, scale=24.0)
    step(r, [1, 1])
    step(r, [4, 1])


@pytest.mark.gpu
def test_repeats_are_bit_identical_and_streams_work():
    import torch
    r = Rows(3, 900, 8, 2, 128, [800, 20, 333], seed=24)
    qkv = r.tokens(3, 9)
    state = r.rng.bit_generator.state
    a = step(r, [1, 9, 5], 4, qkv=qkv, advance=False)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    r.rng.bit_generator.state = state
    with torch.cuda.stream(side):
        b = step(r, [1, 9, 5], 4, qkv=qkv, advance=False, stream=side)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1], equal_nan=True)


@pytest.mark.gpu
def test_captured_call_replays():
    import torch
    r = Rows(2, 500, 8, 2, 64, [400, 33], seed=25)
    q, k, v = r.tokens(2, 1)
    qd, kd, vd = dev(q), dev(k), dev(v)
    acc = torch.rand((2, 2, 500), device="cuda")
    res = torch.zeros_like(acc)
    out = torch.full((2, 1, 8, 64), 12345.0, dtype=torch.bfloat16, device="cuda")
    r.cache.append_weights(0, qd, kd, vd, [1, 1], acc, res, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.cache.append_weights(0, qd, kd, vd, [1, 1], acc, res, out=out)
    for _ in range(2):
        q, k, v = r.tokens(2, 1)
        qd.copy_(dev(q)), kd.copy_(dev(k)), vd.copy_(dev(v))
        was = res.cpu().numpy()
        g.replay()
        torch.cuda.synchronize()
        check(r, 0, [0, 1], [1, 1], q, k, v, None, acc.cpu().numpy(), was, bits_of(out),
              res.cpu().numpy())


@pytest.mark.gpu
def test_refusals_change_nothing():
    import torch
    import kv_cache_incremental_gb300 as kvi
    r = Rows(2, 200, 4, 2, 64, [100, 190], seed=51, kinds=(0, 1), W=8)
    q, k, v = (dev(x) for x in r.tokens(2, 1))
    acc = torch.zeros((2, 2, 200), device="cuda")
    for layer, last in ((1, 1), (0, 0), (0, -1), (2, 1)):
        with pytest.raises(kvi.KVError):
            r.cache.append_weights(layer, q, k, v, [1, 1], acc, acc, last=last)
    with pytest.raises(TypeError):
        r.cache.append_weights(0, q, k, v, [1, 1], acc.half(), acc)
    with pytest.raises(ValueError):
        r.cache.append_weights(0, q, k, v, [1, 1], acc, acc[:1].contiguous())
    with pytest.raises(ValueError):
        r.cache.append_weights(0, q, k, v, [1, 1], acc, acc.cpu())
    big = [dev(x) for x in r.tokens(2, 20)]
    with pytest.raises(kvi.KVCacheFull):
        r.cache.append_weights(0, *big, [1, 20], acc, acc)
    torch.cuda.synchronize()
    assert r.cache.lens == [100, 190] and float(acc.abs().max()) == 0


def test_null_checks_need_no_gpu():
    from kv_cache_incremental_gb300 import _lib
    lib = _lib.load()
    assert lib.kv_append_weights(None, 0, None, None, None, 4, 1, None, None, 0, 1, None, None,
                                 None, None) == 1
