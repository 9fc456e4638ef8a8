"""Plain references, in numpy, of the operators that read a long cache in part.

Keys and queries are taken as the cache holds them (rotated, bf16); scores, softmax and
sums are in 64 bits.  The block choice follows its definition's float32 steps.
"""
from __future__ import annotations

import numpy as np

import oracle

BLOCK = 64
STEP = np.float32(1.0 / 127.0)


def f32(bits):
    return oracle.bf16_to_f32(bits)


def to_bits(x):
    """bf16 bits of a float32 array, round to nearest even (finite values)."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def levels(x):
    """x [..., D] float32 in 127ths of its largest magnitude: (unrounded levels, step)."""
    m = np.abs(x).max(-1).astype(np.float32)
    some = m >= np.float32(1e-30)
    inv = np.where(some, np.float32(127) / np.where(some, m, np.float32(1)), np.float32(0))
    return x * inv[..., None].astype(np.float32), np.where(some, m * STEP, np.float32(0))


def choose(K, q, slot, sink, top_k, recent):
    """Blocks one query reads: K [slots, D] and q [rep, D] float32 (rotated, of one kv head)."""
    nb = slot // BLOCK + 1
    if nb <= sink + top_k + recent:
        return list(range(nb))
    D = K.shape[-1]
    last = nb - recent
    blk = K[:last * BLOCK].reshape(last, BLOCK, D)
    lo, hi = blk.min(1), blk.max(1)
    lev, step = levels(np.concatenate([lo, hi], -1))
    lo8 = np.clip(np.floor(lev[:, :D]), -127, 127).astype(np.int64)
    hi8 = np.clip(np.ceil(lev[:, D:]), -127, 127).astype(np.int64)
    ql, qs = levels(q)
    q8 = np.clip(np.rint(ql), -127, 127).astype(np.int64)
    dot = np.maximum(q8[:, None] * lo8[None], q8[:, None] * hi8[None]).sum(-1)
    score = (dot.astype(np.float32) * (qs[:, None] * step[None]).astype(np.float32)).max(0)
    cand = sorted(range(sink, last), key=lambda b: (-score[b], b))[:top_k]
    return list(range(sink)) + sorted(cand) + list(range(last, nb))


def softmax_attend(K, V, q, visible):
    """q [rep, D], K, V [slots, D] float64, visible [slots] bool: (weights [rep, slots], out
    [rep, D], bound [rep, D] on how far the kernels' output may be off)."""
    D = K.shape[-1]
    s = q @ K.T / np.sqrt(D)
    s = np.where(visible[None], s, -np.inf)
    w = np.exp(s - s.max(-1, keepdims=True))
    w = w / w.sum(-1, keepdims=True)
    out = w @ V
    return w, out, out_bound(q, K, V, w, out)


def score_error(q, K):
    """Largest error [rep] of a score in float32: D products summed in any order (each of the
    at most D additions rounds by half a step of at most the sum of magnitudes), then scaled
    and shifted by the maximum: three more roundings of numbers no larger than twice it."""
    D = K.shape[-1]
    mag = (np.abs(q) @ np.abs(K).T / np.sqrt(D)).max(-1)
    return mag * (D + 8) * 2.0 ** -24


def weight_error(q, K):
    """Largest relative error [rep] of a softmax weight: its score and the maximum are off by
    score_error each, the sum's terms too, exp2 by 2 ulp and the sum of n terms in float32 by
    at most (number of sequential additions, under 512 with the kernels' per-lane sums) half
    steps."""
    return 4 * score_error(q, K) + (512 + 8) * 2.0 ** -24


def out_bound(q, K, V, w, out):
    """The weights' error, their split into two bf16 halves (2^-16 of a weight stays out), the
    float32 sum of up to 512 tile products and partials, and one rounding to bf16 (half a step
    is 2^-8 of the value, at least half the smallest normal's)."""
    mag = w @ np.abs(V)
    rel = weight_error(q, K)[:, None] + 2.0 ** -16 + 512 * 2.0 ** -24
    return 2.0 ** -8 * np.abs(out) + rel * mag * (1 + 2.0 ** -8) + 1e-37


def check_out(got_bits, ref, bound, what=""):
    got = f32(got_bits).astype(np.float64)
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off; first at {i}: got "
                             f"{got[i]!r} want {ref[i]!r} within {bound[i]!r}")


class Rows:
    """A cache of one layout with rows imported from random histories, and what they hold."""

    def __init__(self, B, max_len, Hq, Hk, D, lens, seed=0, kinds=(0,), W=0, paged=False,
                 scale=1.0, K=None, V=None, theta=1e4, blocks=None):
        import kv_cache_incremental_gb300 as kvi
        self.kvi = kvi
        self.rng = np.random.default_rng(seed)
        self.B, self.max_len, self.Hq, self.Hk, self.D = B, max_len, Hq, Hk, D
        self.rep, self.theta, self.kinds, self.W = Hq // Hk, theta, list(kinds), W
        if paged and blocks is None:
            blocks = B * ((max_len + 15) // 16)
        self.cache = kvi.KVCache(B, max_len, Hq, Hk, D, W, list(kinds), theta, 0,
                                 paged_blocks=blocks if paged else None)
        self.K = [[None] * B for _ in kinds]   # [layer][row]: bits [Hk, slots, D]
        self.V = [[None] * B for _ in kinds]
        self.lens = list(lens)
        for b, L in enumerate(lens):
            for l in range(len(kinds)):
                self.K[l][b] = K[l][b] if K else self.bits((Hk, L, D), scale)
                self.V[l][b] = V[l][b] if V else self.bits((Hk, L, D))
            self.fill(b, L)

    def bits(self, shape, scale=1.0):
        return to_bits(self.rng.standard_normal(shape, dtype=np.float32) * np.float32(scale))

    def fill(self, b, L):
        import torch
        parts = []
        for l, kind in enumerate(self.kinds):
            p0 = max(0, L - min(self.W, self.max_len)) if kind == 1 else 0
            parts += [self.K[l][b][:, p0:L].reshape(-1), self.V[l][b][:, p0:L].reshape(-1)]
        flat = np.concatenate(parts) if parts else np.zeros(0, np.uint16)
        buf = dev(flat).view(torch.uint8) if flat.size else torch.empty(16, dtype=torch.uint8,
                                                                        device="cuda")[:0]
        if L > 0:
            self.cache.import_row(b, buf, L)

    def tokens(self, Bs, C, scale=1.0):
        """Random q, k, v bits of a call."""
        return (self.bits((Bs, C, self.Hq, self.D), scale), self.bits((Bs, C, self.Hk, self.D)),
                self.bits((Bs, C, self.Hk, self.D)))

    def rotated(self, x, pos):
        """x bits [n, H, D] rotated at positions pos .. pos + n - 1."""
        p = np.arange(pos, pos + x.shape[0])
        return oracle.rope_bf16(x, p[:, None], self.theta)

    def held(self, layer, b, k, v, pos):
        """Row b's keys and values with the tokens k, v [n, Hk, D] (pre-RoPE) appended."""
        kr = self.rotated(k, pos).transpose(1, 0, 2)
        return (np.concatenate([self.K[layer][b], kr], 1),
                np.concatenate([self.V[layer][b], v.transpose(1, 0, 2)], 1))


def dev(bits):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16).copy())
    return t.view(torch.bfloat16).cuda()


def bits_of(t):
    import torch
    return t.detach().contiguous().cpu().view(torch.int16).numpy().view(np.uint16)
