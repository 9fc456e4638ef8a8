"""Caps in the thousands with scores of a third of the cap up to all of it (kv_append_scored,
kv_append_tree), against 64 bits.

Queries hold powers of two and keys small integers times one, so that every score is an exact
float32 before it is capped, and what is left of the error is the cap's own: the argument and the
tanh within 3 + 8 half steps of the cap, the shift by the maximum (which may run up to 32 log2
units below it) and exp2.  Keys that compete for a query's weight lie in blocks of which some also
hold a score near the cap's other end, so that their caps are taken by different forms; some of
them have one and the same score."""
import numpy as np
import pytest

from scored_ref import lineages
from select_ref import Rows, bits_of, dev, f32, to_bits

E = 2.0 ** -24
THETA = 1e20      # the pairs from D / 4 on turn by less than 1e-7


def vectors(D, coarse, fine, unit):
    """[n, D] with sum `coarse` units over 3D/8 dims and `fine` in one more of the dims that do not
    turn."""
    m = 3 * D // 8
    out = np.zeros((len(coarse), D), np.float32)
    dims = np.r_[D // 4:D // 2, 3 * D // 4:D][:m]
    each, rest = np.divmod(np.abs(coarse), m)
    out[:, dims] = (each[:, None] + (np.arange(m) < rest[:, None])) * np.sign(coarse)[:, None]
    out[:, D - 1] = fine
    return out * np.float32(unit)


def attend(K, V, q, cap, see):
    """q [D], K, V [n, D]: (out, bound)."""
    x = K[see] @ q / np.sqrt(len(q))
    c = cap * np.tanh(x / cap)
    top = c.max()
    # 3 half steps of the argument (the derivative of tanh is at most 1), 8 of the tanh
    err = 3 * E * np.abs(x) + 8 * E * cap + 2 * E * (np.abs(c) + abs(top) + 32) + 2.0 ** -22
    w = np.exp(c - top)
    w = w / w.sum()
    out = w @ V[see]
    rel = np.expm1(err + (w * err).sum() * 1.1) + 2.0 ** -16 + 2 * 520 * E
    return out, 2.0 ** -8 * np.abs(out) + ((w * rel) @ np.abs(V[see])) * (1 + 2.0 ** -8) + 1e-37


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["single", "chunk", "tree"])
@pytest.mark.parametrize("share", [0.35, 0.45, 0.57, 0.85, 0.99])
@pytest.mark.parametrize("cap", [1e3, 3e3, 1e4, 1.6e4, 3e4, 1e5])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_near_a_large_cap(D, cap, share, call):
    import torch
    L, Hk, rep = 700, 2, 4
    rng = np.random.default_rng([int(cap), int(100 * share), D])
    m = 3 * D // 8
    top = m * 100                                     # units of the best keys
    step = cap * share * np.sqrt(D) / top             # of a score before its scale, a unit
    unit, qv = 1.0, np.float32(2.0 ** np.ceil(np.log2(step)))
    # (the rest of the step goes to the share: powers of two on both sides)
    top = int(round(cap * share * np.sqrt(D) / (unit * qv)))
    coarse = rng.integers(-top // 3, top // 3, L)
    fine = np.zeros(L, np.int64)
    best = rng.choice(L, 60, replace=False)           # in every 32 keys a few
    coarse[best] = top
    fine[best[::2]] = rng.integers(0, 12, len(best[::2]))     # half of them equal, half close
    spoil = [j for b in range(0, L, 64) for j in range(b, b + 32) if j not in best][::13]
    coarse[spoil] = -int(0.7 / share * top) if share < 0.7 else -top
    assert np.abs(coarse).max() < 256 * m
    K = np.repeat(to_bits(vectors(D, coarse, fine, unit))[None], Hk, 0)
    V = to_bits(rng.standard_normal((Hk, L, D)).astype(np.float32))
    r = Rows(1, 800, Hk * rep, Hk, D, [L], K=[[K]], V=[[V]], theta=THETA)
    n = 1 if call == "single" else 19
    one = vectors(D, np.array([m]), np.array([2.0 ** -8]), 1.0)[0] * qv
    q = np.stack([one * 2.0 ** -(h % 2) for h in range(Hk * rep)])     # half of the heads at half
    q = to_bits(np.repeat(q[None], n, 0))[None]
    k = np.zeros((1, n, Hk, D), np.uint16)
    v = to_bits(rng.standard_normal((1, n, Hk, D)).astype(np.float32))
    if call == "tree":
        r.cache.enable_tree()
        parents = np.array([-1] + [int(rng.integers(-1, t)) for t in range(1, n)])
        par = torch.from_numpy(parents.astype(np.int32)[None].copy()).cuda()
        out = r.cache.append_tree(0, dev(q), dev(k), dev(v), [n], par, cap=cap)
        seen, pos = lineages(parents), [len(p) - 1 for p in lineages(parents)]
    else:
        out = r.cache.append_scored(0, dev(q), dev(k), dev(v), [n], cap=cap)
        seen, pos = [range(t + 1) for t in range(n)], range(n)
    torch.cuda.synchronize()
    got = f32(bits_of(out))[0].astype(np.float64)
    Kf = np.concatenate([f32(K), np.zeros((Hk, n, D))], 1).astype(np.float64)
    Vf = np.concatenate([f32(V), f32(v[0]).transpose(1, 0, 2)], 1).astype(np.float64)
    for t in range(n):
        qr = f32(r.rotated(q[0, t:t + 1], L + pos[t]))[0].astype(np.float64)
        see = np.arange(L + n) < L
        see[[L + j for j in seen[t]]] = True
        for h in range(Hk * rep):
            x = Kf[h // rep] @ qr[h]
            assert np.array_equal(x, x.astype(np.float32))            # exact, as the bound takes it
            ref, bound = attend(Kf[h // rep], Vf[h // rep], qr[h], cap, see)
            bad = ~(np.abs(got[t, h] - ref) <= bound)
            assert not bad.any(), (t, h, got[t, h][bad][:3], ref[bad][:3], bound[bad][:3])
    assert r.cache.device_error() == 0
