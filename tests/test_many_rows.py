"""Calls of more rows than a 16-bit index counts."""
import numpy as np
import pytest

from select_ref import bits_of

pytestmark = pytest.mark.gpu

B, D = 65600, 64


def inputs(seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((B, 1, 1, D), device="cuda", generator=g).to(torch.bfloat16)
            for _ in range(3)]


@pytest.mark.parametrize("call", ["append", "append_weights", "append_sparse"])
def test_single_token_rows(call):
    """Each row's first token attends to itself alone: the output is its value, its weight 1."""
    import torch
    import kv_cache_incremental_gb300 as kvi
    c = kvi.KVCache(B, 4, 1, 1, D)
    n_new = np.ones(B, dtype=np.int32)
    n_new[1000:64000] = 0                 # two rows of one launch may lie 2^16 apart
    new = torch.from_numpy(n_new == 1).cuda()
    q, k, v = inputs(1)
    out = torch.full_like(q, 12345.0)
    acc = torch.full((B, 1, 4), -3.0, device="cuda")
    if call == "append":
        c.append(0, q, k, v, n_new, out=out)
    elif call == "append_weights":
        c.append_weights(0, q, k, v, n_new, acc, acc, out=out)
        want = torch.where(new, 1.0, -3.0)
        assert torch.equal(acc[:, 0, 0], want) and bool((acc[:, :, 1:] == -3).all())
    else:
        c.enable_sparse(2)
        c.append_sparse(0, q, k, v, n_new, 0, sink=1, recent=1, out=out)
    want = torch.where(new[:, None], v[:, 0, 0], torch.full_like(v[:, 0, 0], 12345.0))
    assert torch.equal(out[:, 0, 0], want)
    K, V = c.storage(0)
    assert torch.equal(V[:, 0, 0], torch.where(new[:, None], v[:, 0, 0], 0))
    assert torch.equal(K[:, 0, 0], torch.where(new[:, None], k[:, 0, 0], 0))  # position 0
    assert c.device_error() == 0
    c.close()


def test_single_token_rows_of_a_hybrid_layer():
    import torch
    import kv_cache_incremental_gb300 as kvi
    c = kvi.KVCache(B, 4, 1, 1, D, 2, [kvi.KV_HYBRID_FULL])
    q, k, v = inputs(2)
    out = torch.full_like(q, 12345.0)
    c.append_hybrid(0, q, k, v, np.ones(B, dtype=np.int32), k_global=k, v_global=v, out=out)
    assert torch.equal(out, v)            # the same key and value twice: half the weight each
    assert torch.equal(c.storage(0)[1][:, 0, 0], v[:, 0, 0])
    assert torch.equal(c.ring_storage(0)[1][:, 0, 0], v[:, 0, 0])
    c.close()
