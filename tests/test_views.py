"""Zero-copy views of a cache's storage keep the cache, and so the memory, alive."""
import gc
import weakref

import pytest

pytestmark = pytest.mark.gpu


def test_views_keep_the_cache_alive():
    import kv_cache_incremental_gb300 as kvi
    c = kvi.KVCache(2, 64, 4, 2, 64, 8, [0, 1])
    ref = weakref.ref(c)
    views = [*c.storage(0), *c.storage(1), c.lpos()]
    del c
    gc.collect()
    assert ref() is not None
    assert all(float(v.float().abs().max()) <= 1 for v in views)    # zeros, and -1 in lpos
    del views
    gc.collect()
    assert ref() is None
