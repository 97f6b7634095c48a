"""The bounds that attention is held to: mistakes planted in the 64-bit form leave them."""

import pytest
import torch

from _attention_bounds import FEW, attention_bounds, few_example, two_parts, way_of
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


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_keys_that_are_rounded_where_they_are_exact(dtype):
    b, cache, q = few_example("single", dtype)
    true = attention_bounds(q, cache, b, dtype=torch.float32)
    assert outside(attention_bounds(q, cache, b, dtype=torch.float32, fault="keys"), true) > 0.1


@pytest.mark.parametrize("name", ["tokens", "drafts"])
def test_weights_in_one_part_where_they_have_two(name):
    b, cache, q = few_example(name, "f16")
    true = attention_bounds(q, cache, b, dtype=torch.float32)
    assert outside(attention_bounds(q, cache, b, dtype=torch.float32, fault="weights"), true) > 0.1


def test_ways_of_sequences():
    for b, heads, kv, d in FEW.values():
        for s in range(b.seqs):
            assert way_of(b, s, heads // kv, torch.float16) == way_of(b, s, heads // kv, torch.bfloat16) == "few"
            assert two_parts(b, "few", heads // kv, d, torch.float16)
            assert not two_parts(b, "few", heads // kv, d, torch.bfloat16)
    b = Batch([100, 100, 100], [1, 16, 17], 16)
    assert [way_of(b, s, 2, torch.float16) for s in range(3)] == ["few", "few", "many"]
    assert [way_of(b, s, 2, torch.float32) for s in range(3)] == ["row"] * 3
