"""Zero-copy views of a cache's storage keep its memory when the cache itself is dropped."""
import gc

import pytest

pytestmark = pytest.mark.gpu


def free_bytes():
    import torch
    torch.cuda.synchronize()
    torch.cuda.empty_cache()      # what torch itself holds but does not use
    return torch.cuda.mem_get_info()[0]


def test_views_keep_the_memory_alive():
    import torch
    import kv_cache_incremental_gb300 as kvi
    torch.zeros(1, device="cuda")
    kvi.KVCache(1, 8, 4, 2, 64).close()                   # contexts, modules
    before = free_bytes()
    c = kvi.KVCache(8, 4096, 4, 4, 128, 8, [0, 1])        # 64 MiB of keys and values
    views = [*c.storage(0), *c.storage(1), c.lpos()]
    again = c.storage(0)
    assert again[0].data_ptr() == views[0].data_ptr()
    held = free_bytes()
    assert before - held > 60 << 20
    del c, again
    gc.collect()
    assert free_bytes() <= held + (1 << 20)               # not freed under the views
    assert all(float(v.float().abs().max()) <= 1 for v in views)    # zeros, and -1 in lpos
    del views
    gc.collect()
    assert free_bytes() - held > 60 << 20


def test_close_frees_at_once_and_twice_is_fine():
    import torch
    import kv_cache_incremental_gb300 as kvi
    torch.zeros(1, device="cuda")
    c = kvi.KVCache(8, 4096, 4, 4, 128)
    view = c.storage(0)
    held = free_bytes()
    c.close()
    c.close()
    assert free_bytes() - held > 60 << 20
    del view, c


def test_a_cache_and_its_graph_collected_together():
    """A reference cycle that holds a cache, a view and a step graph: the collector may
    finalise them in any order."""
    import torch
    import kv_cache_incremental_gb300 as kvi
    torch.zeros(1, device="cuda")
    before = free_bytes()
    for _ in range(3):
        c = kvi.KVCache(8, 4096, 4, 4, 128)
        q = torch.zeros((8, 1, 4, 128), dtype=torch.bfloat16, device="cuda")
        ring = [c.step_graph([q], [q], [q], [q.clone()]), c, c.storage(0)]
        ring.append(ring)
        ring[0].launch()
        torch.cuda.synchronize()
        del c, q, ring
        gc.collect()
    assert before - free_bytes() < 40 << 20
