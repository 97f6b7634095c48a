"""The bounds that attention is held to: mistakes planted in the 64-bit form leave them."""

import pytest
import torch

from _attention_bounds import attention_bounds
from _cache import Batch, random_cache, rows

ONE = Batch([700, 90], [1, 1], 16, single=True)
MANY = Batch([300, 130], [60, 40], 16)


def outside(a, b):
    """The share of a's values outside the bounds of b, by the larger of y's and lse's."""
    out = []
    for i in (0, 2):
        got, want, bound = a[i], b[i], b[i + 1]
        out.append(float((~(((got - want).abs() <= bound) | (got == want))).double().mean()))
    return max(out)


# lse of a single position is its score
SINGLE = Batch([1] * 60, [1] * 60, 16, single=True)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("b,d,softcap", [(SINGLE, 32, 1e3), (ONE, 64, 1e5), (ONE, 64, 1e30), (ONE, 64, 3e38),
                                         (MANY, 64, 1e5), (MANY, 64, 1e30)])
def test_a_cap_that_loses_its_last_bits(dtype, b, d, softcap):
    cache, q = random_cache(1, b.pages, 2, 16, d), rows(2, dtype, b.tokens, 4, d)
    kw = dict(softcap=softcap, dtype=torch.float32)
    true = attention_bounds(q, cache, b, **kw)
    assert outside(attention_bounds(q, cache, b, fault="cap", **kw), true) > 0.01
