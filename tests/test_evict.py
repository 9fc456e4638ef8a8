"""Eviction by accumulated weight (kv_evict_rows, kv_get_slots): the kept slots, the moved
keys, values and accumulators exactly; then every way of going on with an evicted row against
64-bit attention over what it keeps."""
import numpy as np
import pytest

from select_ref import Rows, bits_of, check_out, dev, f32, softmax_attend
import test_sparse
import test_weights


def kept_slots(acc, keep, recent):
    """The definition, one kv head: acc [slots]."""
    n = acc.size
    if n <= keep:
        return np.arange(n)
    old = acc[:n - recent].astype(np.float64)
    old = np.where(np.isnan(old), -np.inf, old)
    nan = np.isnan(acc[:n - recent])
    order = sorted(range(old.size), key=lambda j: (nan[j], -old[j], j))[:keep - recent]
    return np.array(sorted(order) + list(range(n - recent, n)), dtype=np.int64)


def accs(r, seed=0, make=None):
    """An accumulator per global layer: heavy-tailed with ties."""
    rng = np.random.default_rng(seed)
    out = []
    for kind in r.kinds:
        if kind == 1:
            out.append(None)
            continue
        a = (rng.random((r.B, r.Hk, r.max_len), dtype=np.float32) ** 4) * 9
        a[rng.random(a.shape) < 0.15] = 0
        out.append(make(a) if make else a)
    return out


def to_dev(accs_):
    import torch
    return [None if a is None else torch.from_numpy(a.copy()).cuda() for a in accs_]


def expect(src, dst, src_rows, dst_rows, keep, recent, accs_):
    """What dst's rows hold after the eviction: updates dst's bookkeeping; kept per layer."""
    rows = {}
    kept = []
    for l, kind in enumerate(src.kinds):
        kl = []
        for s, d in zip(src_rows, dst_rows):
            K, V = src.K[l][s], src.V[l][s]
            if kind == 1:
                rows[l, d] = (K, V)
                continue
            idx = [kept_slots(accs_[l][s, g, :K.shape[1]], keep, recent) for g in range(src.Hk)]
            rows[l, d] = (np.stack([K[g][i] for g, i in enumerate(idx)]),
                          np.stack([V[g][i] for g, i in enumerate(idx)]))
            kl.append(np.stack(idx))
        kept.append(kl)
    lens = [src.lens[s] for s in src_rows]
    for (l, d), (K, V) in rows.items():
        dst.K[l][d], dst.V[l][d] = K, V
    for d, L in zip(dst_rows, lens):
        dst.lens[d] = L
    return kept


def check_state(r, rows=None):
    """Storage, slots and lengths of rows against the bookkeeping, bit for bit."""
    assert r.cache.lens == r.lens
    slots = r.cache.slots
    for l, kind in enumerate(r.kinds):
        K, V = (bits_of(x) for x in r.cache.storage(l))
        for b in rows if rows is not None else range(r.B):
            n = r.K[l][b].shape[1]
            if kind == 0:
                assert slots[b] == n, (b, slots[b], n)
                at = np.arange(n)
                pos = at
            else:
                pos = np.arange(max(0, r.lens[b] - r.cache.R), r.lens[b])
                at = pos % r.cache.R
            assert np.array_equal(K[b][:, at], r.K[l][b][:, pos]), f"layer {l} row {b}: K"
            assert np.array_equal(V[b][:, at], r.V[l][b][:, pos]), f"layer {l} row {b}: V"
    if r.cache.paged_blocks is not None:
        for b in range(r.B):
            assert len(r.cache.block_table(b)) == (slots[b] + 15) // 16


def evict(src, dst, src_rows, dst_rows, keep, recent, accs_=None, stream=None, alias=False):
    import torch
    accs_ = accs_ or accs(src, seed=keep)
    n = len(src_rows)
    acc_in = to_dev(accs_)
    if alias:
        acc_out = acc_in
    else:
        acc_out = [None if k == 1 else torch.full((dst.B, dst.Hk, dst.max_len), -5.0,
                                                  device="cuda") for k in dst.kinds]
    was = [None if a is None else a.cpu().numpy() for a in acc_out]
    kept = dst.cache.evict_rows(src.cache, src_rows, dst_rows, keep, recent, acc_in,
                                acc_out=acc_out, stream=stream)
    torch.cuda.synchronize()
    want = expect(src, dst, src_rows, dst_rows, keep, recent, accs_)
    for l, kind in enumerate(src.kinds):
        if kind == 1:
            continue
        got, moved = kept[l].cpu().numpy(), acc_out[l].cpu().numpy()
        for i, (s, d) in enumerate(zip(src_rows, dst_rows)):
            m = want[l][i].shape[1]
            assert np.array_equal(got[i][:, :m], want[l][i])
            assert np.all(got[i][:, m:] == -1)
            for g in range(src.Hk):
                assert np.array_equal(moved[d, g, :m], accs_[l][s, g][want[l][i][g]],
                                      equal_nan=True)
                assert np.array_equal(moved[d, g, m:], was[l][d, g, m:], equal_nan=True)
    return kept


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("D,Hk,rep", [(64, 2, 4), (128, 3, 1)])
def test_into_another_cache(D, Hk, rep, paged):
    lens = [0, 1, 99, 100, 101, 640, 1000]
    kw = dict(kinds=(0, 1, 0), W=24, paged=paged)
    src = Rows(7, 1100, Hk * rep, Hk, D, lens, seed=1, **kw)
    dst = Rows(9, 1030, Hk * rep, Hk, D, [5, 50, 0, 700, 0, 0, 3, 64, 9], seed=2, **kw)
    rows = [3, 0, 8, 1, 5, 2, 7]
    evict(src, dst, list(range(7)), rows, 100, 17)
    check_state(dst)
    check_state(src)
    evict(src, dst, [6, 5], [4, 6], 300, 0)
    evict(src, dst, [6, 5], [4, 6], 300, 300)
    evict(src, dst, [2, 4], [1, 0], 1, 0)
    evict(src, dst, [2, 4], [1, 0], 1, 1)
    check_state(dst)


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("alias", [False, True])
def test_in_place(paged, alias):
    lens = [1000, 30, 513, 600, 900]
    r = Rows(5, 1100, 8, 2, 64, lens, seed=3, kinds=(1, 0, 0), W=40, paged=paged)
    evict(r, r, [0, 1, 2, 4], [0, 1, 2, 4], 500, 60, alias=alias)
    check_state(r)
    evict(r, r, [0, 4, 3], [0, 4, 3], 130, 5, alias=alias)
    check_state(r)
    evict(r, r, [0, 3], [1, 2], 77, 5, alias=alias)       # into other rows of the same cache
    check_state(r)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_in_place_long_moves_by_little(D):
    """Kept slots that move by less than a pass of the in-place kernel, and a prefix that
    stays where it is."""
    L = 3000
    r = Rows(2, 3100, 2, 1, D, [L, L], seed=4)
    def make(a):
        a[:] = 5
        a[0, 0, [3, 700, 701, 2500]] = 0                  # few holes
        a[1, 0, :1200] = 7
        a[1, 0, 1200:L:2] = 1                             # every other one goes
        return a
    evict(r, r, [0], [0], L - 4, 10, accs(r, make=make))
    evict(r, r, [1], [1], 2100, 10, accs(r, make=make))
    check_state(r)


@pytest.mark.gpu
def test_orders_of_weights():
    """Ties, negative weights, both zeros, infinities and NaN."""
    def make(a):
        a[0] = 1                                          # all alike: the first ones stay
        a[1, :, :50] = -a[1, :, :50]
        a[2, :, ::3] = 0.0
        a[2, :, 1::3] = -0.0
        a[2, :, 2::3] = np.where(a[2, :, 2::3] > 1, 1e-40, -1e-40)
        a[3, :, 7::9] = np.nan
        a[3, :, 8::9] = np.inf
        a[3, :, 5::9] = -np.inf
        a[4] = np.nan
        return a
    r = Rows(6, 400, 4, 2, 64, [300, 300, 300, 300, 300, 300], seed=5)
    d = Rows(6, 400, 4, 2, 64, [0] * 6, seed=6)
    evict(r, d, list(range(6)), list(range(6)), 120, 11, accs(r, make=make))
    check_state(d)
    evict(r, d, list(range(6)), list(range(6)), 290, 11, accs(r, make=make))
    check_state(d)


@pytest.mark.gpu
def test_rows_longer_than_shared_memory_holds():
    L = 60000
    r = Rows(1, 61000, 1, 1, 64, [L], seed=7)
    d = Rows(1, 61000, 1, 1, 64, [0], seed=8)
    evict(r, d, [0], [0], 4000, 100)
    check_state(d)
    evict(r, d, [0], [0], 59000, 7)
    check_state(d)


@pytest.mark.gpu
def test_more_items_than_a_launch_holds():
    B = 140
    r = Rows(B, 64, 2, 1, 64, [40 + b % 20 for b in range(B)], seed=9, kinds=(0, 0))
    evict(r, r, list(range(B)), list(range(B)), 33, 4)
    check_state(r)


@pytest.mark.gpu
def test_paged_rows_that_share_a_prefix():
    """Cutting a row in place leaves the rows it shares blocks with as they were."""
    r = Rows(4, 700, 4, 2, 64, [300, 0, 0, 90], seed=10, kinds=(0, 0), paged=True, blocks=100)
    r.cache.copy_rows(r.cache, [0, 0], [1, 2], keep=[300, 210])
    for l in range(2):
        r.K[l][1], r.V[l][1] = r.K[l][0], r.V[l][0]
        r.K[l][2], r.V[l][2] = r.K[l][0][:, :210], r.V[l][0][:, :210]
    r.lens = [300, 300, 210, 90]
    check_state(r)
    free = r.cache.free_blocks
    evict(r, r, [0], [0], 64, 8)
    check_state(r)
    assert r.cache.free_blocks == free - 4 + 1            # four copies; its own last block back
    evict(r, r, [1, 2], [1, 2], 100, 8)
    check_state(r)
    evict(r, r, [1], [3], 50, 8)
    check_state(r)
    used = sum(len(r.cache.block_table(b)) for b in range(4))
    assert r.cache.free_blocks == 100 - used


@pytest.mark.gpu
def test_pool_exhaustion_changes_nothing():
    import kv_cache_incremental_gb300 as kvi
    r = Rows(3, 200, 4, 2, 64, [100, 0, 0], seed=11, paged=True, blocks=8)
    r.cache.copy_rows(r.cache, [0], [1])
    r.K[0][1], r.V[0][1], r.lens[1] = r.K[0][0], r.V[0][0], 100
    assert r.cache.free_blocks == 0                       # 7 and a copied last one
    acc = to_dev(accs(r))
    with pytest.raises(kvi.KVPoolExhausted):
        r.cache.evict([0], 40, 5, acc)                    # copies of three shared blocks
    with pytest.raises(kvi.KVPoolExhausted):
        r.cache.evict_rows(r.cache, [0], [2], 40, 5, acc)
    check_state(r)


@pytest.mark.gpu
@pytest.mark.parametrize("D,paged", [(64, False), (64, True), (128, False), (128, True)])
def test_going_on_with_evicted_rows(D, paged):
    """After an eviction the other calls append at the next slot, rotate at the true position
    and attend to what is kept: dense decode and chunks, the step graph, sparse and counted
    calls, another eviction, reset, import and copies into the row."""
    import torch
    import kv_cache_incremental_gb300 as kvi
    r = Rows(4, 900, 8, 2, D, [700, 300, 64, 500], seed=12, paged=paged)
    r.cache.enable_sparse(5)
    test_sparse.step(r, [1, 1, 1, 1], 1, 2, 2)
    evict(r, r, [0, 1, 3], [0, 1, 3], 200, 30)
    assert r.cache.lens == [701, 301, 65, 501] and r.cache.slots == [200, 200, 65, 200]
    dense_step(r, [1, 1, 1, 1])
    dense_step(r, [70, 1, 5, 33])
    dense_step(r, [2, 0, 64, 1])
    test_sparse.step(r, [1, 66, 1, 2], 1, 2, 2)
    test_weights.step(r, [1, 3, 1, 40], 2)
    test_weights.step(r, [1, 1, 1, 1])
    graph_step(r)
    evict(r, r, [0, 1], [0, 1], 150, 30)
    test_sparse.step(r, [1, 1, 1, 1], 1, 1, 1)
    graph_step(r)
    check_state(r)
    for call in (lambda: r.cache.copy_rows(r.cache, [0], [2]),
                 lambda: r.cache.copy_rows(r.cache, [0], [0], keep=[10]),
                 lambda: r.cache.export_row(0)):
        with pytest.raises(kvi.KVError):
            call()
    check_state(r)
    # ordinary again
    r.cache.reset([0])
    r.K[0][0] = r.V[0][0] = np.zeros((2, 0, D), np.uint16)
    r.lens[0] = 0
    r.cache.copy_rows(r.cache, [2], [1])
    r.K[0][1], r.V[0][1], r.lens[1] = r.K[0][2], r.V[0][2], r.lens[2]
    r.K[0][3], r.V[0][3], r.lens[3] = r.bits((2, 40, D)), r.bits((2, 40, D)), 40
    r.fill(3, 40)
    dense_step(r, [30, 1, 1, 1])
    test_sparse.step(r, [1, 1, 1, 66], 1, 1, 1)
    check_state(r)
    assert r.cache.slots == r.cache.lens and r.cache.device_error() == 0


def dense_step(r, n_new):
    import torch
    C = max(n_new)
    q, k, v = r.tokens(r.B, C)
    out = torch.full((r.B, C, r.Hq, r.D), 12345.0, dtype=torch.bfloat16, device="cuda")
    r.cache.append(0, dev(q), dev(k), dev(v), n_new, out=out)
    r.cache.advance(n_new)
    torch.cuda.synchronize()
    check_dense(r, n_new, q, k, v, bits_of(out))


def check_dense(r, n_new, q, k, v, got):
    for b, n in enumerate(n_new):
        assert np.all(got[b, n:] == np.uint16(0x4641))
        if n == 0:
            continue
        K, V = r.held(0, b, k[b, :n], v[b, :n], r.lens[b])
        qr = f32(r.rotated(q[b, :n], r.lens[b])).reshape(n, r.Hk, r.rep, r.D).astype(np.float64)
        for t in range(n):
            m = K.shape[1] - n + t + 1
            for g in range(r.Hk):
                _, ref, bound = softmax_attend(f32(K[g, :m]).astype(np.float64),
                                               f32(V[g, :m]).astype(np.float64), qr[t, g],
                                               np.ones(m, bool))
                check_out(got[b, t, g * r.rep:(g + 1) * r.rep], ref, bound,
                          f"row {b} token {t} head {g}")
        r.K[0][b], r.V[0][b] = K, V
        r.lens[b] += n


def graph_step(r):
    import torch
    q, k, v = r.tokens(r.B, 1)
    bufs = [[dev(x)] for x in (q, k, v)]
    out = torch.full((r.B, 1, r.Hq, r.D), 12345.0, dtype=torch.bfloat16, device="cuda")
    g = r.cache.step_graph(*bufs, [out])
    g.launch()
    torch.cuda.synchronize()
    check_dense(r, [1] * r.B, q, k, v, bits_of(out))
    g.close()


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
def test_a_step_graph_made_before_the_eviction(paged):
    import torch
    r = Rows(3, 400, 8, 2, 64, [300, 90, 17], seed=13, paged=paged)
    q, k, v = r.tokens(3, 1)
    qd, kd, vd = dev(q), dev(k), dev(v)
    out = torch.empty_like(qd)
    g = r.cache.step_graph([qd], [kd], [vd], [out])
    for keep in (None, 64, 40):
        if keep:
            evict(r, r, [0, 1], [0, 1], keep, 9)
        q, k, v = r.tokens(3, 1)
        qd.copy_(dev(q)), kd.copy_(dev(k)), vd.copy_(dev(v))
        out.fill_(12345.0)
        g.launch()
        torch.cuda.synchronize()
        check_dense(r, [1] * 3, q, k, v, bits_of(out))
    check_state(r)
    g.close()


@pytest.mark.gpu
def test_shared_blocks_are_counted_once():
    """Two rows cut in place that hold the same blocks: one of them keeps the originals, so
    copies for the other are all the pool has to give."""
    r = Rows(2, 64, 4, 2, 64, [48, 0], seed=14, paged=True, blocks=5)
    r.cache.copy_rows(r.cache, [0], [1])
    r.K[0][1], r.V[0][1], r.lens[1] = r.K[0][0], r.V[0][0], 48
    assert r.cache.free_blocks == 2
    evict(r, r, [0, 1], [0, 1], 32, 3)
    check_state(r)
    assert r.cache.free_blocks == 1


@pytest.mark.gpu
def test_sliding_and_global_layers_keep_their_own_positions():
    """Two layers: after an eviction the sliding one still goes by positions (ring slots,
    window, rotation), the global one by slots."""
    import torch
    from harness import Scenario
    a = Scenario(B=2, max_len=400, Hq=4, Hk=2, D=64, W=16, kinds=[1, 0], seed=61)
    b = Scenario(B=2, max_len=400, Hq=4, Hk=2, D=64, W=16, kinds=[1, 0], seed=61)
    for sc in (a, b):
        for n in ([64, 50], [64, 64], [30, 64]):
            sc.step(n, C=64, check=False)
    acc = torch.rand((2, 2, 400), device="cuda")
    a.cache.evict([0, 1], 100, 20, [None, acc])
    for n, C in (([1, 1], 1), ([20, 7], 20), ([1, 1], 1)):
        oa = a.step(n, C=C, check=False)
        ob = b.step(n, C=C, check=False)
        x, y = bits_of(oa[0][1]), bits_of(ob[0][1])       # the sliding layer: unaffected
        assert np.array_equal(x, y)
    assert np.array_equal(a.cache.lpos().cpu().numpy(), b.cache.lpos().cpu().numpy())
    for x, y in zip(a.cache.storage(0), b.cache.storage(0)):
        assert np.array_equal(bits_of(x)[:, :, :16], bits_of(y)[:, :, :16])


@pytest.mark.gpu
def test_generation_within_a_budget():
    """The operators together, as a serving loop uses them: a prompt whose last queries are
    counted, counted decode steps, eviction whenever a row reaches its limit, sparse steps in
    between; a side stream throughout."""
    import torch
    r = Rows(3, 600, 8, 2, 64, [0, 0, 0], seed=71, paged=True)
    r.cache.enable_sparse(4)
    side = torch.cuda.Stream()
    rng = np.random.default_rng(3)
    acc = torch.full((3, 2, 600), float("nan"), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        def counted(n_new, last=None):
            C = max(n_new)
            q, k, v = r.tokens(3, C)
            before = acc.cpu().numpy()
            out = torch.full((3, C, 8, 64), 12345.0, dtype=torch.bfloat16, device="cuda")
            r.cache.append_weights(0, dev(q), dev(k), dev(v), n_new, acc, acc, last=last, out=out,
                                   stream=side)
            torch.cuda.synchronize()
            test_weights.check(r, 0, [0, 1, 2], n_new, q, k, v, last, before, before,
                               bits_of(out), acc.cpu().numpy())
            r.cache.advance(n_new, stream=side)
            for b, n in enumerate(n_new):
                r.K[0][b], r.V[0][b] = r.held(0, b, k[b, :n], v[b, :n], r.lens[b])
                r.lens[b] += n
        counted([130, 70, 20], 16)
        for i in range(12):
            counted([1, 1, 1])
            over = [b for b in range(3) if r.cache.slots[b] > 80]
            if over:
                now = [acc.cpu().numpy()]
                kept = r.cache.evict(over, 64, 16, [acc], stream=side)
                torch.cuda.synchronize()
                want = expect(r, r, over, over, 64, 16, now)
                for i, b in enumerate(over):
                    assert np.array_equal(kept[0].cpu().numpy()[i], want[0][i])
            if i % 4 == 3:
                test_sparse.step(r, [1, 1, 1], 0, 1, 1, stream=side)
                # a step that is not counted: its own key starts at no weight
                for b in range(3):
                    acc[b, :, r.cache.slots[b] - 1] = 0
        check_state(r)
    assert r.cache.device_error() == 0


@pytest.mark.gpu
def test_two_caches_on_two_streams_at_once():
    """Calls of two caches queued on two streams with nothing waiting between them."""
    import torch
    rs = [Rows(3, 900, 8, 2, 64, [800, 300, 500], seed=90 + i, paged=i == 1) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in rs]
    work = []
    for r in rs:
        r.cache.enable_sparse(4)
        qkv = [[dev(x) for x in r.tokens(3, 1)] for _ in range(3)]
        acc = torch.rand((3, 2, 900), device="cuda")
        work.append((qkv, acc))
    torch.cuda.synchronize()
    results = [[], []]
    for turn in range(2):           # in turn, then alone: the same results
        if turn == 1:
            rs = [Rows(3, 900, 8, 2, 64, [800, 300, 500], seed=90 + i, paged=i == 1)
                  for i in range(2)]
            for r in rs:
                r.cache.enable_sparse(4)
            torch.cuda.synchronize()
        accs_ = [w[1].clone() for w in work]
        torch.cuda.synchronize()
        outs = [[], []]
        for step in range(3):
            for i, r in enumerate(rs):
                s, (q, k, v) = streams[i], work[i][0][step]
                if step == 0:
                    o = r.cache.append_weights(0, q, k, v, [1] * 3, accs_[i], accs_[i], stream=s)
                elif step == 1:
                    r.cache.evict([0, 2], 200, 30, [accs_[i]], stream=s)
                    o = r.cache.append_sparse(0, q, k, v, [1] * 3, 1, stream=s)
                else:
                    o = r.cache.append(0, q, k, v, [1] * 3, stream=s)
                r.cache.advance([1] * 3, stream=s)
                outs[i].append(o)
                if turn == 1:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        for i in range(2):
            results[turn].append([bits_of(o) for o in outs[i]] + [accs_[i].cpu().numpy()])
    for a, b in zip(*results):
        for x, y in zip(a, b):
            assert np.array_equal(x, y)


@pytest.mark.gpu
def test_refusals_change_nothing():
    import torch
    import kv_cache_incremental_gb300 as kvi
    r = Rows(3, 200, 4, 2, 64, [100, 150, 60], seed=51, kinds=(0, 1), W=8)
    acc = to_dev(accs(r))
    ev = r.cache.evict_rows
    bad = [((r.cache, [0], [0], 0, 0, acc), {}),            # keep
           ((r.cache, [0], [0], 201, 0, acc), {}),
           ((r.cache, [0], [0], 10, 11, acc), {}),          # recent
           ((r.cache, [0], [0], 10, -1, acc), {}),
           ((r.cache, [0], [3], 10, 1, acc), {}),           # rows
           ((r.cache, [-1], [0], 10, 1, acc), {}),
           ((r.cache, [0, 1], [2, 2], 10, 1, acc), {}),
           ((r.cache, [0, 1], [1, 2], 10, 1, acc), {}),     # 1 is written and read
           ((r.cache, [0, 0], [0, 1], 10, 1, acc), {})]
    for args, kw in bad:
        with pytest.raises(kvi.KVError):
            ev(*args, **kw)
    with pytest.raises(ValueError):
        ev(r.cache, [0], [0], 10, 1, [None, None])
    with pytest.raises(ValueError):
        ev(r.cache, [0], [0], 10, 1, acc[:1])
    with pytest.raises(TypeError):
        ev(r.cache, [0], [0], 10, 1, [acc[0].double(), None])
    other = kvi.KVCache(3, 200, 4, 2, 64, 9, [0, 1])
    with pytest.raises(kvi.KVError):
        other.evict_rows(r.cache, [0], [0], 10, 1, acc)     # another window
    short = kvi.KVCache(3, 120, 4, 2, 64, 8, [0, 1])
    with pytest.raises(kvi.KVError):
        short.evict_rows(r.cache, [1], [0], 10, 1, acc)     # 150 positions
    hy = kvi.KVCache(1, 64, 4, 2, 64, 8, [2, 3])
    with pytest.raises(kvi.KVError):
        hy.evict([0], 10, 1, [None, None])
    sl = kvi.KVCache(1, 64, 4, 2, 64, 8, [1])
    with pytest.raises(kvi.KVError):
        sl.evict([0], 10, 1, [None])
    check_state(r)


def test_null_checks_need_no_gpu():
    from kv_cache_incremental_gb300 import _lib
    lib = _lib.load()
    assert lib.kv_evict_rows(None, None, None, None, 0, 1, 0, None, None, None, None) == 1
    assert lib.kv_get_slots(None, None) == 1


def test_reference_choice_on_a_worked_example():
    a = np.array([5, 1, 3, 3, 0, 9], np.float32)
    assert kept_slots(a, 4, 1).tolist() == [0, 2, 3, 5]
    assert kept_slots(a, 3, 1).tolist() == [0, 2, 5]
    assert kept_slots(a, 6, 1).tolist() == [0, 1, 2, 3, 4, 5]
    assert kept_slots(np.array([np.nan, -np.inf, 1], np.float32), 2, 0).tolist() == [1, 2]
