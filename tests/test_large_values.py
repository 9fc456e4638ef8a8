"""Values near the end of bf16's range: a token's output is a mean of values, and finite where the
sum of 2^(x - m) V over its keys, m its largest score, is a float32 (as in kv_append).  Scores
rise from one block of the chunk kernel to the next, or from one tile of the decode kernel to the
next, by less than what makes their running maxima move, so that a weight taken of the running
maximum would be up to 2^14 or 2^7.5."""
import numpy as np
import pytest

from scored_ref import attend, lineages
from select_ref import Rows, bits_of, check_out, dev, f32, to_bits
from test_large_caps import THETA, vectors

L = 1500


def log2_scores(form):
    j = np.arange(L)
    if form == "tiles":                                # 64 keys at 0, 64 at 7.5
        return np.where(j // 64 % 2 == 1, 7.5, 0.0)
    if form == "pairs":                                # 128 keys at 24 behind 128 at 0
        return np.where(j // 128 % 2 == 0, 24.0, 0.0)
    return np.interp(j, [0, 500, L], [28.0, 0.0, 14.0])      # blocks go the newest first


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["single", "chunk", "tree"])
@pytest.mark.parametrize("change", ["none", "cap", "slopes", "first"])
@pytest.mark.parametrize("form", ["tiles", "blocks", "pairs"])
@pytest.mark.parametrize("D", [64, 128])
def test_values_near_the_largest(D, form, change, call):
    import torch
    if call == "tree" and change == "first":
        pytest.skip("a tree has no first positions")
    Hk, rep, m = 2, 4, 3 * D // 8
    rng = np.random.default_rng([D, len(form), len(change)])
    qv = 2.0 ** -4
    cap, slopes, first = 0.0, None, None
    x = log2_scores(form) * np.log(2)
    if change == "cap":
        cap = 40.0
        x = cap * np.arctanh(x / cap)
    K = np.repeat(to_bits(vectors(D, np.rint(x * np.sqrt(D) / qv).astype(np.int64),
                                  np.zeros(L), 1.0))[None], Hk, 0)
    V = np.ldexp(1 + rng.random((Hk, L, D)), 115).astype(np.float32)     # up to 2^116
    V[:, :, ::4] *= rng.choice([-1, 1], V[:, :, ::4].shape)
    V = to_bits(V)
    plain = to_bits(rng.standard_normal((2, Hk, L, D)).astype(np.float32))
    r = Rows(2, 1600, Hk * rep, Hk, D, [L, L], K=[[K, plain[0]]], V=[[V, plain[1]]], theta=THETA)
    n = 1 if call == "single" else 21
    q = to_bits(np.broadcast_to(vectors(D, np.array([m]), np.zeros(1), 1.0)[0] * np.float32(qv),
                                (2, n, Hk * rep, D)))
    k = np.zeros((2, n, Hk, D), np.uint16)
    v = to_bits(np.ldexp(rng.random((2, n, Hk, D)), 115).astype(np.float32))
    kw = dict(cap=cap)
    if change == "slopes":
        slopes = np.float32(2.0 ** -np.arange(12, 20))
        kw["slopes"] = torch.from_numpy(slopes).cuda()
    if change == "first":
        first = np.full((2, n), 37)
        kw["first"] = torch.from_numpy(first.astype(np.int32)).cuda()
    if call == "tree":
        r.cache.enable_tree()
        parents = np.array([-1] + [int(rng.integers(-1, t)) for t in range(1, n)])
        par = torch.from_numpy(np.stack([parents] * 2).astype(np.int32)).cuda()
        out = r.cache.append_tree(0, dev(q), dev(k), dev(v), [n, n], par, **kw)
        seen, pos = lineages(parents), [len(p) - 1 for p in lineages(parents)]
    else:
        out = r.cache.append_scored(0, dev(q), dev(k), dev(v), [n, n], **kw)
        seen, pos = [range(t + 1) for t in range(n)], list(range(n))
    torch.cuda.synchronize()
    got = bits_of(out)
    for b in range(2):
        Kf = np.concatenate([f32(r.K[0][b]), np.zeros((Hk, n, D))], 1).astype(np.float64)
        Vf = np.concatenate([f32(r.V[0][b]), f32(v[b]).transpose(1, 0, 2)], 1).astype(np.float64)
        at = np.r_[np.arange(L), L + np.array(pos)]
        for t in range(n):
            qr = f32(r.rotated(q[b, t:t + 1], L + pos[t]))[0].astype(np.float64)
            see = np.arange(L + n) < L
            see[[L + j for j in seen[t]]] = True
            if first is not None:
                see &= at >= first[b, t]
            for g in range(Hk):
                h = slice(g * rep, (g + 1) * rep)
                ref, bound = attend(Kf[g], Vf[g], qr[h], L + pos[t] - at, see, cap,
                                    None if slopes is None else slopes[h])
                check_out(got[b, t, h], ref, bound, f"row {b} token {t} head {g}")
    assert r.cache.device_error() == 0
