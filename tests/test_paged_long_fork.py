"""A fork of a paged row with more blocks than one block-table launch writes (2048): every
entry of the new row's table reaches the device."""
import numpy as np
import pytest

from harness import torch_to_bits
from select_ref import Rows, dev

pytestmark = pytest.mark.gpu


def test_fork_of_a_row_of_more_than_2048_blocks():
    import torch
    L = 2048 * 16 + 40
    r = Rows(2, L + 10, 2, 1, 64, [L, 0], seed=1, paged=True, blocks=2100)
    r.cache.copy_rows(r.cache, [0], [1])
    assert r.cache.block_table(1)[:2050] == r.cache.block_table(0)[:2050]
    q, k, v = (dev(np.repeat(x, 2, 0)) for x in r.tokens(1, 1))
    out = torch.empty_like(q)
    r.cache.append(0, q, k, v, [1, 1], out=out)       # both rows hold the same keys
    a, b = torch_to_bits(out)
    assert np.array_equal(a, b)
