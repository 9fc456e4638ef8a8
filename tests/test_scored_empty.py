"""Chunks with changed scores whose keys are split so that some query tiles have no block in a piece:
early tiles of a prompt, documents of fewer blocks than pieces, tokens that see nothing.  Such a
CTA issues no product, and leaves nothing behind that could arrive after its end: the CTAs that
follow it on its SM, and their barriers, are the ones that would be written."""
import numpy as np
import pytest

from scored_ref import Scored
from select_ref import bits_of, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,rep", [(64, 4), (128, 4), (128, 16)])
@pytest.mark.parametrize("what", ["prompt", "documents", "nothing"])
def test_pieces_without_blocks(D, rep, what):
    import torch
    r = Scored(3, 1100, rep, 1, D, [0, 130, 3], seed=71)
    n, C = [900, 40, 300], 900
    first = None
    if what == "documents":
        first = np.stack([np.arange(C) // 130 * 130] * 3)
    elif what == "nothing":
        first = np.full((3, C), 1 << 20)
    qkv = r.tokens(3, C)
    got = r.call(n, cap=9.0, first=first, qkv=qkv, advance=False)
    fi = None if first is None else torch.from_numpy(first.astype(np.int32)).cuda()
    q, k, v = (dev(x) for x in qkv)
    outs = [torch.full((3, C, rep, D), 12345.0, dtype=torch.bfloat16, device="cuda")
            for _ in range(20)]
    for out in outs:                       # back to back, each on the heels of the one before
        r.cache.append_scored(0, q, k, v, n, cap=9.0, first=fi, out=out)
    torch.cuda.synchronize()
    for out in outs:
        assert np.array_equal(bits_of(out), got)
    assert r.cache.device_error() == 0
