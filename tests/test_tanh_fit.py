"""The polynomials of a capped score (score_mod.cuh), as written there in float32, against tanh."""
import os
import re

import numpy as np
import pytest

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir,
                      "kv_cache_incremental_gb300", "csrc", "score_mod.cuh")


@pytest.mark.parametrize("name,limit,error", [("tanh_coef", "kTanhSmall", 7.5e-8),
                                              ("tanh_coef3", "kTanhTiny", 6.7e-8)])
def test_largest_relative_error(name, limit, error):
    with open(SOURCE) as f:
        text = f.read()
    c = re.search(name + r"\(int i\) \{\s*constexpr float c\[\d\] = \{([^}]*)\}", text).group(1)
    c = [float(np.float32(x.strip().rstrip("f"))) for x in c.split(",")]
    top = float(re.search(limit + r" = ([0-9.]+)f;", text).group(1))
    x = np.linspace(1e-4, top, 200001)
    off = np.abs(x * np.polyval(c[::-1], x * x) / np.tanh(x) - 1).max()
    assert error - 1e-9 < off < error + 5e-10          # what the comment states
