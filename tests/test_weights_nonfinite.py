"""Accumulated weights beside keys with infinite components: a key that every query scores
-inf weighs nothing and adds nothing, whatever the number of counted query vectors -- the
kernels take them in groups of 8 and 16 and fill up the last one."""
import numpy as np
import pytest

from select_ref import (Rows, bits_of, check_out, dev, f32, softmax_attend, to_bits,
                        weight_error)

INF = np.uint16(0x7F80)


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("Hk,rep,D,n_new,last", [
    (2, 4, 64, [3, 1, 9], None),        # 12, 4 and 36 counted vectors
    (2, 1, 128, [5, 17, 70], None),     # 5, 17, 64 and 6
    (1, 7, 64, [30, 2, 1], 3),          # 21, 14, 7
    (1, 16, 128, [2, 66, 1], 5),        # whole groups
    (2, 3, 64, [7, 40, 2], 1),          # 3: one group, all but empty
])
def test_keys_that_score_minus_infinity(Hk, rep, D, n_new, last, paged):
    import torch
    lens = [500, 290, 131]
    B, d = 3, D // 2 - 1                # the slowest pair: rotated by less than 0.08
    r = Rows(B, 640, Hk * rep, Hk, D, lens, seed=D + rep, paged=paged)
    dead = [[0, 77, 300, L - 1] if L > 300 else [5, 64, L - 1] for L in lens]
    for b, L in enumerate(lens):
        r.K[0][b][:, dead[b], d] = INF
        r.fill(b, L)
    C = max(n_new)
    q, k, v = r.tokens(B, C)
    qf = f32(q)
    qf[..., d] = -1 - np.abs(qf[..., d])
    q = to_bits(qf)                     # rotated: below -1 cos 0.08 + 6 sin 0.08 < 0
    before = r.rng.random((B, Hk, 640), dtype=np.float32)
    acc_in = torch.from_numpy(before.copy()).cuda()
    acc_out = torch.full_like(acc_in, -3.0)
    out = torch.full((B, C, Hk * rep, D), 12345.0, dtype=torch.bfloat16, device="cuda")
    r.cache.append_weights(0, dev(q), dev(k), dev(v), n_new, acc_in, acc_out, last=last, out=out)
    torch.cuda.synchronize()
    got, acc = bits_of(out), acc_out.cpu().numpy()
    for b, n in enumerate(n_new):
        L, counted = lens[b], n if last is None else min(n, last)
        K, V = r.held(0, b, k[b, :n], v[b, :n], L)
        qr = f32(r.rotated(q[b, :n], L)).reshape(n, Hk, rep, D).astype(np.float64)
        assert qr[..., d].max() < 0
        Kf, Vf = f32(K).astype(np.float64), f32(V).astype(np.float64)
        Kf[:, dead[b]] = 0              # the reference leaves these keys out
        for g in range(Hk):
            want = np.zeros(L + n)
            want[:L] = before[b, g, :L]
            slack = np.abs(want) * 2.0 ** -24
            for t in range(n):
                m = L + t + 1
                vis = np.ones(m, bool)
                vis[dead[b]] = False
                w, ref, bound = softmax_attend(Kf[g, :m], Vf[g, :m], qr[t, g], vis)
                check_out(got[b, t, g * rep:(g + 1) * rep], ref, bound, f"row {b} token {t}")
                if t >= n - counted:
                    want[:m] += w.sum(0)
                    slack[:m] += (w * weight_error(qr[t, g], Kf[g, :m])[:, None]).sum(0)
            slack += want * (counted * rep + 2) * 2.0 ** -24 + 1e-37
            mine = acc[b, g, :L + n].astype(np.float64)
            assert np.array_equal(mine[dead[b]], want[dead[b]]), (b, g, mine[dead[b]])
            assert np.all(np.abs(mine - want) <= slack), (b, g)
    assert r.cache.device_error() == 0
