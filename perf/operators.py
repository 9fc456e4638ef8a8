"""What the operators that let a long cache be read in part are measured on.

Three operators of the cache, each over dense and paged caches:

  sparse   append a step's tokens and attend, for every query token and kv head, to the
           first ``sink`` blocks of 64 keys, the last ``recent`` ones and the ``top_k``
           others whose 8-bit key bounds promise the largest score (KVCache.append_sparse)
  weights  append and attend to everything, and add the softmax weights of the step's
           (last) queries to a per-key accumulator (KVCache.append_weights)
  evict    keep a row's last ``recent`` keys and its heaviest others by that accumulator,
           and make a row of the kept keys (KVCache.evict_rows)

``run`` computes each operator with elementary torch operations, or with ``own`` set
through this repository's package.  ``exact`` gives the same in 64 bits.
"""
import math

import numpy as np
import torch

own = False

THETA = 1e4
BLOCK = 64


# ---------------------------------------------------------------------------- cases
def listed():
    # The shapes are the ones this repository tests and benchmarks: the small sliding/global
    # layout (Hq 8, Hk 2, D 64), the decode-bandwidth one (B 64, Hq 32, Hk 8, D 128, 1k-8k),
    # the long-context one (B 16, Hq 64, Hk 8, D 128, 16k-32k) and the continuous batch
    # (Hq 16, Hk 4, D 64, right-padded chunks of 64).
    small = dict(Hq=8, Hk=2, D=64)
    decode = dict(Hq=32, Hk=8, D=128)
    long = dict(Hq=64, Hk=8, D=128)
    cont = dict(Hq=16, Hk=4, D=64)
    return [
        # one user's next token after a short document: what a call costs at the least
        dict(name="sparse_one_row", op="sparse", B=1, lo=1990, hi=1990, max_len=2048, C=1,
             sink=1, top_k=8, recent=2, paged=False, **small),
        # a full decode batch of ordinary contexts
        dict(name="sparse_decode", op="sparse", B=64, lo=1024, hi=8190, max_len=8192, C=1,
             sink=1, top_k=16, recent=2, paged=False, **decode),
        # long documents in a paged cache: scoring the blocks weighs against reading them
        dict(name="sparse_long", op="sparse", B=16, lo=16384, hi=32766, max_len=32768, C=1,
             sink=1, top_k=32, recent=4, paged=True, **long),
        # the next turn's prompt, cut into right-padded chunks, beside rows that decode
        dict(name="sparse_chunk", op="sparse", B=24, lo=0, hi=12000, max_len=16384, C=64,
             sink=1, top_k=16, recent=2, paged=False, **cont),
        # the first steps of a short conversation with its weights counted
        dict(name="weights_one_row", op="weights", B=1, lo=299, hi=299, max_len=512, C=1,
             last=1, paged=False, **small),
        # a decode batch that counts every step's weights
        dict(name="weights_decode", op="weights", B=64, lo=1024, hi=8190, max_len=8192, C=1,
             last=1, paged=False, **decode),
        # the same over long documents in a paged cache
        dict(name="weights_long", op="weights", B=16, lo=16384, hi=32766, max_len=32768, C=1,
             last=1, paged=True, **long),
        # a prompt's chunks whose last 32 queries say which keys matter
        dict(name="weights_chunk", op="weights", B=24, lo=0, hi=12000, max_len=16384, C=64,
             last=32, paged=False, **cont),
        # one short row cut to its budget
        dict(name="evict_one_row", op="evict", B=1, lo=700, hi=700, max_len=1024, keep=256,
             recent=33, kinds="0", W=0, paged=False, **small),
        # a batch of rows cut after their prompts, sliding and global layers
        dict(name="evict_batch", op="evict", B=32, lo=1024, hi=8190, max_len=8192, keep=1024,
             recent=128, kinds="10", W=512, paged=False, **decode),
        # long documents of a paged cache, the six-layer period of the long-context layout
        dict(name="evict_long", op="evict", B=8, lo=16384, hi=32766, max_len=32768, keep=4096,
             recent=512, kinds="111110", W=512, paged=True, **long),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sparse", "weights", "evict"])
    Hk = rng.choice([1, 2, 3, 4, 8])
    D = rng.choice([64, 128])
    rep = rng.choice([1, 2, 3, 4, 7, 8, 16])
    if Hk * rep > 64:
        rep = 8
    case = dict(op=op, Hq=Hk * rep, Hk=Hk, D=D, paged=rng.random() < 0.4)
    C = 1 if rng.random() < 0.6 or op == "evict" else _log_int(rng, 2, 90)
    B = _log_int(rng, 1, 64)
    top = _log_int(rng, 100, 32000)
    # key bytes and score work of the whole call, kept below the largest listed case
    while B * Hk * D * top > 64 * 8 * 128 * 5000 or B * C * Hk * rep * top > 24 * 64 * 16 * 8000:
        if B > 1 and (top < 1000 or rng.random() < 0.5):
            B = max(1, B // 2)
        elif top > 100:
            top = max(100, top // 2)
        else:
            C = max(1, C // 2)
    if C > 1 and B * C > 1536:
        B = max(1, 1536 // C)
    case.update(B=B, lo=rng.randint(0 if op != "evict" else 1, top), hi=top,
                max_len=top + C + rng.randint(0, 40))
    if op == "evict":
        keep = _log_int(rng, 1, max(2, top))
        case.update(keep=keep, recent=rng.randint(0, keep), kinds=rng.choice(["0", "00", "10"]),
                    W=rng.choice([5, 64, 500]))
    else:
        case["C"] = C
    if op == "sparse":
        case.update(sink=rng.randint(0, 2), top_k=_log_int(rng, 1, 40), recent=rng.randint(1, 4))
    if op == "weights":
        case["last"] = rng.randint(1, C)
    return case


def _lens_and_new(case):
    """Cached tokens and new tokens of every row: a fixed function of the case."""
    rng = np.random.default_rng([case["B"], case["hi"], case.get("C", 0), case["D"]])
    lens = rng.integers(case["lo"], case["hi"] + 1, size=case["B"])
    C = case.get("C", 0)
    if C <= 1:
        return lens.tolist(), [C] * case["B"]
    n_new = rng.integers(0, C + 1, size=case["B"])
    n_new[rng.random(case["B"]) < 0.2] = 1      # rows in their decode phase
    n_new[0] = C
    return lens.tolist(), n_new.tolist()


def work(case):
    Hq, Hk, D, B = case["Hq"], case["Hk"], case["D"], case["B"]
    lens, n_new = _lens_and_new(case)
    by = fl = 0
    if case["op"] == "evict":
        for k in case["kinds"]:
            for L in lens:
                kept = min(L, case["keep"]) if k == "0" else min(L, case["W"])
                by += 2 * 2 * kept * Hk * D * 2           # K and V, read and written
                if k == "0":
                    by += Hk * (4 * L + 4 * kept + 4 * case["keep"])   # weights in, out, kept
        return {"bytes": by, "flops": fl}
    for L, n in zip(lens, n_new):
        if n == 0:
            continue
        by += n * (2 * Hq + 4 * Hk) * D * 2               # q, k, v in; new K, V and out
        if case["op"] == "weights":
            by += 2 * (L + n) * Hk * D * 2 + Hk * 4 * (2 * (L + n) - n)
            for t in range(n):
                fl += 4 * (L + t + 1) * Hq * D
        else:
            # every key that some query of the row attends to is read once: at least one
            # query's selection, at most the whole row
            per = case["sink"] + case["top_k"] + case["recent"]
            most = 0
            for t in range(n):
                nb = (L + t) // BLOCK + 1
                keys = min(L + t + 1, per * BLOCK)
                most = max(most, keys)
                fl += 4 * keys * Hq * D
                if nb > per:
                    fl += 2 * 2 * (nb - case["sink"] - case["recent"]) * Hq * D
                by += Hk * 4 * per                        # the selected blocks
            by += 2 * most * Hk * D * 2
            nb = (L + n - 1) // BLOCK + 1
            if nb > per:
                by += (nb - case["sink"] - case["recent"]) * Hk * (2 * D + 4)
    return {"bytes": by, "flops": fl}


# ---------------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    return g


def _history(case, lens, g, first=0):
    """Post-RoPE keys and values of the cached positions, [B, Hk, max_len, D] bf16, zero past
    each row's length.  Keys lean towards a per-head direction by an amount that differs from
    block to block, so that some blocks matter more, as they do in text."""
    B, Hk, D, M = case["B"], case["Hk"], case["D"], case["max_len"]
    lean = _direction(case, g)
    K = torch.zeros((B, Hk, M, D), dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    nb = (M + BLOCK - 1) // BLOCK
    gain = torch.randn((B, Hk, nb), generator=g, device="cuda") * 0.6
    for b in range(B):
        L = lens[b]
        x = torch.randn((Hk, L, D), generator=g, device="cuda")
        x += lean[:, None, :] * gain[b].repeat_interleave(BLOCK, dim=1)[:, :L, None]
        K[b, :, :L] = x.to(torch.bfloat16)
        V[b, :, :L] = torch.randn((Hk, L, D), generator=g, device="cuda").to(torch.bfloat16)
    return K, V, lean


def _direction(case, g):
    Hk, D = case["Hk"], case["D"]
    lean = torch.randn((Hk, D), generator=g, device="cuda")
    low = torch.zeros(D, device="cuda")     # the slowly turning half of the rotary pairs
    low[D // 4:D // 2] = 1
    low[3 * D // 4:] = 1
    return lean * low


def _inputs(case, seed):
    """Everything a program holds before the call, as plain tensors."""
    g = _generator(seed)
    lens, n_new = _lens_and_new(case)
    B, Hq, Hk, D, M = case["B"], case["Hq"], case["Hk"], case["D"], case["max_len"]
    st = dict(case=case, lens=lens, n_new=n_new)
    if case["op"] == "evict":
        st["K"], st["V"], st["acc"] = [], [], []
        for kind in case["kinds"]:
            K, V, _ = _history(case, lens, g)
            st["K"].append(K)
            st["V"].append(V)
            if kind == "0":
                # accumulated weights fall off steeply, and keys that never drew any tie at 0
                a = torch.rand((B, Hk, M), generator=g, device="cuda")
                a = torch.where(a < 0.1, torch.zeros_like(a), (a * a * a * a) * 20)
                st["acc"].append(a)
            else:
                st["acc"].append(None)
        return st
    K, V, lean = _history(case, lens, g)
    C = case["C"]
    q = torch.randn((B, C, Hq, D), generator=g, device="cuda")
    q += lean.repeat_interleave(Hq // Hk, dim=0)
    st.update(K=K, V=V, q=q.to(torch.bfloat16),
              k=torch.randn((B, C, Hk, D), generator=g, device="cuda").to(torch.bfloat16),
              v=torch.randn((B, C, Hk, D), generator=g, device="cuda").to(torch.bfloat16))
    if case["op"] == "weights":
        st["acc_in"] = torch.rand((B, Hk, M), generator=g, device="cuda") * 3
    return st


def _rope_table(pos, D):
    """cos, sin [len(pos), D / 2] float32, of angles taken in double."""
    inv = np.array([THETA ** ((-2.0 * i) / D) for i in range(D // 2)])
    a = np.asarray(pos, dtype=np.float64)[:, None] * inv[None, :]
    return (torch.from_numpy(np.cos(a).astype(np.float32)).cuda(),
            torch.from_numpy(np.sin(a).astype(np.float32)).cuda())


def _import_rows(cache, case, lens, Ks, Vs):
    """Fill a cache's rows from plain histories through its public import."""
    Hk, D = case["Hk"], case["D"]
    for b, L in enumerate(lens):
        if L == 0:
            continue
        parts = []
        for K, V, kind in zip(Ks, Vs, case.get("kinds", "0")):
            p0 = max(0, L - min(case["W"], case["max_len"])) if kind == "1" else 0
            parts += [K[b, :, p0:L].reshape(-1), V[b, :, p0:L].reshape(-1)]
        cache.import_row(b, torch.cat(parts).view(torch.uint8), L)


def prepare(case, seed):
    st = _inputs(case, seed)
    B, Hq, Hk, D, M = case["B"], case["Hq"], case["Hk"], case["D"], case["max_len"]
    lens, n_new = st["lens"], st["n_new"]
    if case["op"] == "evict":
        n_glob = case["kinds"].count("0")
        st["kept"] = [torch.full((B, Hk, case["keep"]), -1, dtype=torch.int32, device="cuda")
                      if k == "0" else None for k in case["kinds"]]
        st["acc_out"] = [torch.zeros((B, Hk, M), device="cuda") if k == "0" else None
                         for k in case["kinds"]]
        assert n_glob >= 1
    else:
        C = case["C"]
        st["out"] = torch.zeros((B, C, Hq, D), dtype=torch.bfloat16, device="cuda")
        if case["op"] == "sparse":
            per = case["sink"] + case["top_k"] + case["recent"]
            st["selected"] = torch.full((B, C, Hk, per), -1, dtype=torch.int32, device="cuda")
        else:
            st["acc_out"] = torch.zeros((B, Hk, M), device="cuda")
        # the rotary table is a plan that a program keeps
        st["rope"] = [_rope_table(range(L, L + n), D) for L, n in zip(lens, n_new)]
    if own:
        import kv_cache_incremental_gb300 as kvi
        kinds = [int(k) for k in case.get("kinds", "0")]
        pool = B * ((M + 15) // 16) if case["paged"] else None
        cache = kvi.KVCache(B, M, Hq, Hk, D, case.get("W", 0), kinds, THETA, 0,
                            paged_blocks=pool)
        Ks = st["K"] if case["op"] == "evict" else [st["K"]]
        Vs = st["V"] if case["op"] == "evict" else [st["V"]]
        _import_rows(cache, case, lens, Ks, Vs)
        st["cache"] = cache
        if case["op"] == "sparse":
            cache.enable_sparse(case["sink"] + case["top_k"] + case["recent"])
            cache.update_sparse(0)       # the prompt's block bounds, kept like its keys
        if case["op"] == "evict":        # the rows of kept keys are built in a cache of their own
            st["dst"] = kvi.KVCache(B, M, Hq, Hk, D, case.get("W", 0), kinds, THETA, 0)
        st["K"] = st["V"] = None
    elif case["op"] == "evict":
        st["dK"] = [torch.zeros((B, Hk, case["keep"], D), dtype=torch.bfloat16, device="cuda")
                    if k == "0" else _ring_shape(case) for k in case["kinds"]]
        st["dV"] = [torch.zeros_like(x) for x in st["dK"]]
    elif case["op"] == "sparse":
        nb = (M + BLOCK - 1) // BLOCK    # bounds of the cached blocks, kept like the keys
        st["bmin"] = torch.zeros((B, Hk, nb, D), dtype=torch.int8, device="cuda")
        st["bmax"] = torch.zeros_like(st["bmin"])
        st["bscale"] = torch.zeros((B, Hk, nb), device="cuda")
        for b, L in enumerate(lens):
            _bounds_plain(st, b, 0, L // BLOCK)
    torch.cuda.synchronize()
    return st


def _ring_shape(case):
    R = min(case["W"], case["max_len"])
    return torch.zeros((case["B"], case["Hk"], R, case["D"]), dtype=torch.bfloat16, device="cuda")


# ---------------------------------------------------------------------------- plain forms
def _rope_plain(x, cs):
    """Half-split rotation of x [n, H, D] by (cos, sin) [n, D / 2], rounded to bf16."""
    c, s = cs[0][:, None, :], cs[1][:, None, :]
    h = x.shape[-1] // 2
    x1, x2 = x[..., :h].float(), x[..., h:].float()
    return torch.cat([x1 * c - x2 * s, x1 * s + x2 * c], dim=-1).to(torch.bfloat16)


def _append_plain(st, b):
    """Row b's new keys and values at positions lens .. lens + n - 1; its rotated queries."""
    L, n = st["lens"][b], st["n_new"][b]
    cs = st["rope"][b]
    st["K"][b, :, L:L + n] = _rope_plain(st["k"][b, :n], cs).transpose(0, 1)
    st["V"][b, :, L:L + n] = st["v"][b, :n].transpose(0, 1)
    return _rope_plain(st["q"][b, :n], cs)


def _bounds_plain(st, b, b0, b1):
    """8-bit bounds of blocks [b0, b1) of row b: the scale is a 127th of the block's largest
    magnitude, the lower bound rounds down and the upper one up."""
    if b1 <= b0:
        return
    K = st["K"][b, :, b0 * BLOCK:b1 * BLOCK].float()
    K = K.reshape(K.shape[0], b1 - b0, BLOCK, K.shape[-1])
    lo, hi = K.amin(2), K.amax(2)
    big = torch.maximum(lo.abs(), hi.abs()).amax(-1)
    ok = big >= 1e-30
    inv = torch.where(ok, torch.full_like(big, 127.0) / torch.where(ok, big, 1.0), 0.0)
    st["bmin"][b, :, b0:b1] = torch.floor(lo * inv[..., None]).clamp(-127, 127).to(torch.int8)
    st["bmax"][b, :, b0:b1] = torch.ceil(hi * inv[..., None]).clamp(-127, 127).to(torch.int8)
    st["bscale"][b, :, b0:b1] = torch.where(ok, big * (1.0 / 127.0), 0.0)


def _select_plain(st, b, q):
    """Blocks each of row b's new queries reads, [n, Hk, per] ascending, -1 past the last."""
    case = st["case"]
    sink, top_k, recent = case["sink"], case["top_k"], case["recent"]
    L, n, Hk = st["lens"][b], st["n_new"][b], case["Hk"]
    per = sink + top_k + recent
    qf = q.float().reshape(n, Hk, -1, case["D"])
    big = qf.abs().amax(-1)
    ok = big >= 1e-30
    inv = torch.where(ok, torch.full_like(big, 127.0) / torch.where(ok, big, 1.0), 0.0)
    qi = torch.round(qf * inv[..., None]).clamp(-127, 127)
    qs = torch.where(ok, big * (1.0 / 127.0), 0.0)
    nb_all = (L + n - 1) // BLOCK + 1
    lo = st["bmin"][b, :, :nb_all].float()
    hi = st["bmax"][b, :, :nb_all].float()
    # sum over the head of max(q lo, q hi): whole numbers below 2^24, so float32 sums are exact
    dot = (torch.einsum("nhrd,hbd->nhrb", qi.clamp(min=0), hi)
           + torch.einsum("nhrd,hbd->nhrb", qi.clamp(max=0), lo))
    score = (dot * (qs[..., None] * st["bscale"][b, None, :, None, :nb_all])).amax(2)
    nb = (torch.arange(L, L + n, device="cuda") // BLOCK + 1)[:, None, None]
    idx = torch.arange(nb_all, device="cuda")
    exists = idx < nb
    always = exists & ((idx < sink) | (idx >= nb - recent))
    cand = exists & ~always
    order = torch.sort(torch.where(cand, score, -torch.inf), dim=-1, descending=True,
                       stable=True)[1]
    rank = torch.empty_like(order)
    rank.scatter_(-1, order, torch.arange(nb_all, device="cuda").expand_as(order).contiguous())
    take = always | (cand & (rank < top_k))
    key = torch.where(take, idx, nb_all + idx)
    key = torch.sort(key, dim=-1)[0][..., :per]
    out = torch.full((n, Hk, per), -1, dtype=torch.int32, device="cuda")
    out[..., :key.shape[-1]] = torch.where(key < nb_all, key, -1).to(torch.int32)
    return out, take


def _attend_plain(st, b, q, visible):
    """Softmax weights [Hk, rep, n, slots] of row b's queries over its visible keys, and the
    attention outputs [n, Hq, D]."""
    case = st["case"]
    L, n, Hk, D = st["lens"][b], st["n_new"][b], case["Hk"], case["D"]
    K, V = st["K"][b, :, :L + n].float(), st["V"][b, :, :L + n].float()
    qf = q.float().reshape(n, Hk, -1, D).permute(1, 2, 0, 3)
    s = torch.matmul(qf, K[:, None].transpose(-1, -2)) * (1.0 / math.sqrt(D))
    s = torch.where(visible, s, -torch.inf)
    w = torch.exp(s - s.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    o = torch.matmul(w, V[:, None])
    return w, o.permute(2, 0, 1, 3).reshape(n, case["Hq"], D)


def _causal(L, n):
    return (torch.arange(L + n, device="cuda")[None, :]
            <= torch.arange(L, L + n, device="cuda")[:, None])


def _sparse_plain(st):
    case = st["case"]
    for b in range(case["B"]):
        L, n = st["lens"][b], st["n_new"][b]
        if n == 0:
            continue
        q = _append_plain(st, b)
        _bounds_plain(st, b, L // BLOCK, (L + n) // BLOCK)
        sel, take = _select_plain(st, b, q)
        st["selected"][b, :n] = sel
        vis = take.repeat_interleave(BLOCK, dim=-1)[..., :L + n] & _causal(L, n)[:, None, :]
        _, o = _attend_plain(st, b, q, vis.transpose(0, 1)[:, None])
        st["out"][b, :n] = o.to(torch.bfloat16)
    return _outputs(st, st["selected"], st["K"], st["V"])


def _weights_plain(st):
    case = st["case"]
    for b in range(case["B"]):
        L, n = st["lens"][b], st["n_new"][b]
        if n == 0:
            continue
        q = _append_plain(st, b)
        w, o = _attend_plain(st, b, q, _causal(L, n))
        st["out"][b, :n] = o.to(torch.bfloat16)
        add = w[:, :, max(0, n - case["last"]):].sum((1, 2))
        add[:, :L] += st["acc_in"][b, :, :L]
        st["acc_out"][b, :, :L + n] = add
    return _outputs(st, st["acc_out"], st["K"], st["V"])


def _evict_plain(st):
    case = st["case"]
    keep, recent = case["keep"], case["recent"]
    outs = []
    for l, kind in enumerate(case["kinds"]):
        K, V = st["K"][l], st["V"][l]
        for b, L in enumerate(st["lens"]):
            if kind == "1":
                R = min(case["W"], case["max_len"])
                p = torch.arange(max(0, L - R), L, device="cuda")
                st["dK"][l][b, :, p % R] = K[b, :, p]
                st["dV"][l][b, :, p % R] = V[b, :, p]
                continue
            m = min(L, keep)
            if L <= keep:
                idx = torch.arange(L, device="cuda").expand(case["Hk"], L)
            else:
                a = st["acc"][l][b, :, :L - recent]
                heavy = torch.sort(a, dim=-1, descending=True, stable=True)[1][:, :keep - recent]
                last = torch.arange(L - recent, L, device="cuda").expand(case["Hk"], recent)
                idx = torch.sort(torch.cat([heavy, last], dim=-1), dim=-1)[0]
            rows = idx[..., None].expand(-1, -1, case["D"])
            st["dK"][l][b, :, :m] = torch.gather(K[b], 1, rows)
            st["dV"][l][b, :, :m] = torch.gather(V[b], 1, rows)
            st["acc_out"][l][b, :, :m] = torch.gather(st["acc"][l][b], 1, idx)
            st["kept"][l][b, :, :m] = idx.to(torch.int32)
        outs += [st["dK"][l], st["dV"][l]]
        if kind == "0":
            outs += [st["acc_out"][l], st["kept"][l]]
    return outs


def _outputs(st, second, K, V):
    """A step's outputs: the attention, the selection or the weights, and the updated keys and
    values where they lie in one place (a paged cache spreads them over its pool's blocks)."""
    outs = [st["out"], second]
    return outs if st["case"]["paged"] else outs + [K, V]


# ---------------------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"sparse": _sparse_plain, "weights": _weights_plain, "evict": _evict_plain}[op](st)
    cache = st["cache"]
    if op == "evict":
        dst = st["dst"]
        dst.evict_rows(cache, list(range(case["B"])), list(range(case["B"])), case["keep"],
                       case["recent"], st["acc"], acc_out=st["acc_out"], kept=st["kept"])
        outs = []
        for l, kind in enumerate(case["kinds"]):
            K, V = dst.storage(l)
            m = case["keep"] if kind == "0" else min(case["W"], case["max_len"])
            outs += [K[:, :, :m], V[:, :, :m]]   # the rows' live slots, views of the storage
            if kind == "0":
                outs += [st["acc_out"][l], st["kept"][l]]
        return outs
    if op == "sparse":
        cache.append_sparse(0, st["q"], st["k"], st["v"], st["n_new"], case["top_k"],
                            sink=case["sink"], recent=case["recent"], out=st["out"],
                            selected=st["selected"])
        second = st["selected"]
    else:
        cache.append_weights(0, st["q"], st["k"], st["v"], st["n_new"], st["acc_in"],
                             st["acc_out"], last=case["last"], out=st["out"])
        second = st["acc_out"]
    if case["paged"]:
        return _outputs(st, second, None, None)
    K, V = cache.storage(0)
    M = case["max_len"]
    return _outputs(st, second, K[:, :, :M], V[:, :, :M])


# ---------------------------------------------------------------------------- 64 bits
def _exact_rotated(x, pos):
    """Rotated vectors as the cache holds them.  bfloat16 keys and queries are what the
    operators are defined on, so this step rounds as the definition does: float32 products,
    one float32 sum, bfloat16."""
    D = x.shape[-1]
    ang = [[p * THETA ** ((-2.0 * i) / D) for i in range(D // 2)] for p in pos]
    c = torch.tensor([[math.cos(a) for a in r] for r in ang], dtype=torch.float32).cuda()[:, None]
    s = torch.tensor([[math.sin(a) for a in r] for r in ang], dtype=torch.float32).cuda()[:, None]
    a, b = x.float().split(D // 2, dim=-1)
    lo = torch.sub(torch.mul(a, c), torch.mul(b, s))
    hi = torch.add(torch.mul(a, s), torch.mul(b, c))
    return torch.cat((lo, hi), -1).bfloat16().double()


def _levels(x):
    """x in 127ths of its largest magnitude along the last axis: (levels before rounding,
    step).  The definition takes these in float32."""
    m = x.float().abs().max(-1, keepdim=True).values
    tiny = m < 1e-30
    safe = torch.where(tiny, torch.ones_like(m), m)
    lev = x.float() * torch.div(torch.full_like(safe, 127.0), safe)
    return (torch.where(tiny, torch.zeros_like(lev), lev),
            torch.where(tiny, torch.zeros_like(m), m * np.float32(1.0 / 127.0).item())[..., 0])


def _exact_blocks(case, K, L, q, t):
    """The set of blocks, per kv head, that token t (at slot L + t) reads; q [Hk, rep, D]."""
    sink, top_k, recent = case["sink"], case["top_k"], case["recent"]
    nb = (L + t) // BLOCK + 1
    if nb <= sink + top_k + recent:
        return [list(range(nb))] * case["Hk"]
    last = nb - recent
    full = K[:, :last * BLOCK].reshape(case["Hk"], last, BLOCK, -1)
    low, high = full.min(2).values, full.max(2).values
    both = torch.cat([low, high], -1)
    lev, step = _levels(both)
    D = case["D"]
    low8 = lev[..., :D].floor().clamp(-127, 127).double()
    high8 = lev[..., D:].ceil().clamp(-127, 127).double()
    qlev, qstep = _levels(q)
    q8 = qlev.round().clamp(-127, 127).double()
    sets = []
    for h in range(case["Hk"]):
        best = None
        for r in range(q.shape[1]):
            v = q8[h, r]
            dot = torch.maximum(v * low8[h], v * high8[h]).sum(-1)
            sc = dot.float() * (qstep[h, r] * step[h])
            best = sc if best is None else torch.maximum(best, sc)
        best = best.cpu().numpy()
        cand = sorted(range(sink, last), key=lambda i: (-best[i], i))[:top_k]
        sets.append(sorted(list(range(sink)) + cand + list(range(last, nb))))
    return sets


def exact(case, seed):
    """The outputs of run in 64 bits."""
    st = _inputs(case, seed)
    if case["op"] == "evict":
        return _exact_evict(case, st)
    B, C, Hq, Hk, D, M = (case[x] for x in ("B", "C", "Hq", "Hk", "D", "max_len"))
    total = sum(st["n_new"])
    if case["op"] == "sparse" and total * Hq > 30000:
        return None     # token by token and head by head: too slow for the largest chunks
    out = torch.zeros((B, C, Hq, D), dtype=torch.float64, device="cuda")
    if case["op"] == "sparse":
        per = case["sink"] + case["top_k"] + case["recent"]
        second = torch.full((B, C, Hk, per), -1, dtype=torch.int64, device="cuda")
    else:
        second = torch.zeros((B, Hk, M), dtype=torch.float64, device="cuda")
    for b, (L, n) in enumerate(zip(st["lens"], st["n_new"])):
        if n == 0:
            continue
        q = _exact_rotated(st["q"][b, :n], range(L, L + n)).reshape(n, Hk, Hq // Hk, D)
        new = _exact_rotated(st["k"][b, :n], range(L, L + n))
        st["K"][b, :, L:L + n] = new.permute(1, 0, 2).bfloat16()
        st["V"][b, :, L:L + n] = st["v"][b, :n].permute(1, 0, 2)
        K, V = st["K"][b, :, :L + n].double(), st["V"][b, :, :L + n].double()
        if case["op"] == "weights":
            total_w = torch.zeros((Hk, L + n), dtype=torch.float64, device="cuda")
            total_w[:, :L] = st["acc_in"][b, :, :L].double()
        for t in range(n):
            m = L + t + 1
            logit = torch.einsum("hrd,hkd->hrk", q[t], K[:, :m]) / math.sqrt(D)
            if case["op"] == "sparse":
                sets = _exact_blocks(case, K, L, q[t], t)
                hide = torch.ones((Hk, m), dtype=torch.bool, device="cuda")
                for h, blocks in enumerate(sets):
                    second[b, t, h, :len(blocks)] = torch.tensor(blocks)
                    for j in blocks:
                        hide[h, j * BLOCK:(j + 1) * BLOCK] = False
                logit = logit.masked_fill(hide[:, None], -math.inf)
            p = torch.softmax(logit, -1)
            out[b, t] = torch.einsum("hrk,hkd->hrd", p, V[:, :m]).reshape(Hq, D)
            if case["op"] == "weights" and t >= n - case["last"]:
                total_w[:, :m] += p.sum(1)
        if case["op"] == "weights":
            second[b, :, :L + n] = total_w
    return [out, second] if case["paged"] else [out, second, st["K"], st["V"]]


def _exact_evict(case, st):
    keep, recent, Hk = case["keep"], case["recent"], case["Hk"]
    outs = []
    for l, kind in enumerate(case["kinds"]):
        src = (st["K"][l], st["V"][l])
        if kind == "1":
            R = min(case["W"], case["max_len"])
            ring = [torch.zeros((case["B"], Hk, R, case["D"]), dtype=torch.float64,
                                device="cuda") for _ in src]
            for b, L in enumerate(st["lens"]):
                for slot in range(min(R, L)):
                    p = slot + (L - 1 - slot) // R * R
                    for d, s in zip(ring, src):
                        d[b, :, slot] = s[b, :, p].double()
            outs += ring
            continue
        rows = [torch.zeros((case["B"], Hk, keep, case["D"]), dtype=torch.float64,
                            device="cuda") for _ in src]
        acc = torch.zeros((case["B"], Hk, case["max_len"]), dtype=torch.float64, device="cuda")
        kept = torch.full((case["B"], Hk, keep), -1, dtype=torch.int64, device="cuda")
        weights = st["acc"][l].cpu().numpy()
        for b, L in enumerate(st["lens"]):
            for h in range(Hk):
                if L > keep:
                    w = weights[b, h, :L - recent]
                    heavy = np.lexsort((np.arange(w.size), -w.astype(np.float64)))
                    sel = np.sort(np.concatenate([heavy[:keep - recent],
                                                  np.arange(L - recent, L)]))
                else:
                    sel = np.arange(L)
                i = torch.from_numpy(sel.astype(np.int64)).cuda()
                for d, s in zip(rows, src):
                    d[b, h, :i.numel()] = s[b, h].index_select(0, i).double()
                acc[b, h, :i.numel()] = st["acc"][l][b, h].index_select(0, i).double()
                kept[b, h, :i.numel()] = i
        outs += rows + [acc, kept]
    return outs
