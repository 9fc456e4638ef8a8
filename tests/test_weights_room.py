"""The memory of accumulated weights: a cache's first call that counts them may be a captured
one, and caches that count none hold no room for it."""
import numpy as np
import pytest

from select_ref import Rows, bits_of, dev
import test_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("C", [1, 5])
def test_the_first_call_is_captured(C):
    import torch
    lens = [700, 33]
    test_weights.step(Rows(2, 800, 8, 2, 64, lens, seed=1), [1, C])   # kernels are loaded
    r = Rows(2, 800, 8, 2, 64, lens, seed=2)
    n_new = [1, C]
    q, k, v = r.tokens(2, C)
    qd, kd, vd = dev(q), dev(k), dev(v)
    acc = torch.rand((2, 2, 800), device="cuda")
    res = torch.full_like(acc, -3.0)
    out = torch.full((2, C, 8, 64), 12345.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.cache.append_weights(0, qd, kd, vd, n_new, acc, res, out=out)
    for _ in range(2):
        q, k, v = r.tokens(2, C)
        qd.copy_(dev(q)), kd.copy_(dev(k)), vd.copy_(dev(v))
        was = res.cpu().numpy()
        g.replay()
        torch.cuda.synchronize()
        test_weights.check(r, 0, [0, 1], n_new, q, k, v, None, acc.cpu().numpy(), was,
                           bits_of(out), res.cpu().numpy())
    test_weights.step(r, n_new)                        # and a call beside the graph
    del g
    assert r.cache.device_error() == 0


def test_an_ordinary_cache_holds_no_room_for_scores():
    """Rows whose scores would take 159 MB beside 80 MB of prefill partials."""
    import torch
    import kv_cache_incremental_gb300 as kvi

    def free():
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        return torch.cuda.mem_get_info()[0]

    torch.zeros(1, device="cuda")
    B, L, Hq, Hk, D = 16, 32768, 64, 4, 128
    kvi.KVCache(1, 8, 4, 2, 64).close()                # contexts, modules
    before = free()
    c = kvi.KVCache(B, L, Hq, Hk, D)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    kv = 2 * B * Hk * (L + 1) * D * 2
    rest = 2 * B * Hk * 64 * D * 2 + L * D * 4 + (B * 32 * Hq + min(1024 * sms, B * Hq * 1024)) * (
        D * 4 + 8)
    assert before - free() <= kv + rest + (16 << 20)   # allocations are rounded up
    c.close()


@pytest.mark.parametrize("Hk,rep,D", [(2, 4, 64), (2, 2, 128), (1, 16, 128)])
def test_chunks_whose_last_token_stands_alone(Hk, rep, D):
    """A first call whose rows end in a sub-chunk of one token, the only one counted: nothing is
    read that the attention has not left."""
    r = Rows(3, 800, Hk * rep, Hk, D, [300, 0, 129], seed=6)
    test_weights.step(r, [65, 129, 1], 1)
    test_weights.step(r, [65, 1, 193], 2)
