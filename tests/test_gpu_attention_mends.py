"""Attention over the paged Q4_0 cache at calls that once went wrong."""

import math

import pytest
import torch

from _attention_bounds import FEW, attention_bounds, few_example
from _cache import TYPES, Batch, check, random_cache, rows

pytestmark = pytest.mark.gpu

# (batch, heads, kv heads, d): one position; one row each, cut and not; drafts in products of 16 and of 32
# rows; prompts; both in one batch
WAYS = {
    "single": (Batch([1] * 60, [1] * 60, 16, seed=1, single=True), 4, 2, 32),
    "tokens": (Batch([5000, 700, 1], [1] * 3, 16, single=True), 8, 2, 128),
    "whole": (Batch([100, 400, 7], [1] * 3, 16, seed=3, single=True), 40, 2, 64),
    "drafts": (Batch([900, 1300, 40], [5, 2, 3], 16, seed=4), 10, 2, 128),
    "prompts": (Batch([150, 400], [150, 90], 128, seed=6), 4, 4, 64),
    "mixed": (Batch([900, 700, 300], [1, 50, 120], 16, seed=5, before=1, behind=3), 4, 1, 96),
    "wide": (Batch([330, 90], [100, 1], 32, seed=7), 4, 2, 256),
}


def example(name, dtype, seed=1):
    b, heads, kv, d = WAYS[name]
    return b, random_cache(seed, b.pages, kv, b.page, d), rows(seed + 1, dtype, b.tokens, heads, d)


def same(q4lib, gpu, b, cache, q, what, y_dtype=None, **kw):
    y = torch.full(q.shape, 7.0, dtype=y_dtype or q.dtype, device=gpu)
    lse = torch.full(q.shape[:2], 7.0, device=gpu)
    q4lib.q4_attention(q.to(gpu), torch.from_numpy(cache).to(gpu), *b.device(gpu), return_lse=True, y=y, lse=lse, **kw)
    want, bound, big, lbound = attention_bounds(q, cache, b, dtype=y.dtype, **kw)
    check(y, want, bound, what)
    check(lse, big, lbound, "lse " + what)


# ------------------------------------------------------------------ caps

@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("name", WAYS)
@pytest.mark.parametrize("softcap", [1e-40, 1e-3, 0.7, 30.0, 1e3, 1e6, 1e30, 3e38])
def test_caps_of_every_size(q4lib, gpu, dtype, name, softcap):
    """A cap far above the scores leaves them as they are, one far below makes them all alike;
    rows whose scores reach a cap of 1000 beside rows whose scores are some few."""
    b, cache, q = example(name, dtype)
    for row, _, _ in b.places[::3]:
        q[row, 1] *= 1000
    same(q4lib, gpu, b, cache, q, f"{dtype} {name} cap {softcap}", softcap=softcap)


# ------------------------------------------------------------------ rows that are no numbers

@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("name", WAYS)
@pytest.mark.parametrize("kw", [dict(), dict(scale=0.0), dict(scale=-0.3, window=40), dict(softcap=20.0),
                                dict(scale=0.0, softcap=1e6)])
def test_nan_and_infinities_in_q(q4lib, gpu, dtype, name, kw):
    """One of them anywhere in a row and head of q is NaN in its y and lse, whatever the scale and
    the cap, also where the row sees a single position; other rows and heads have the same bits."""
    b, cache, q = example(name, dtype)
    args = [torch.from_numpy(cache).to(gpu)] + b.device(gpu)
    mine = torch.zeros(q.shape[:2], dtype=torch.bool, device=gpu)
    for row, _, _ in b.places:
        mine[row] = True
    want = q4lib.q4_attention(q.to(gpu), *args, return_lse=True, **kw)
    for i, bad in enumerate((math.nan, math.inf, -math.inf)):
        x, others = q.clone(), mine.clone()
        hit = [(b.places[j][0], (j + i) % q.shape[1]) for j in {0, len(b.places) // 2, len(b.places) - 1}]
        for row, head in hit:
            x[row, head, (row + 5 * i) % q.shape[2]] = bad
            others[row, head] = False
        y, lse = q4lib.q4_attention(x.to(gpu), *args, return_lse=True, **kw)
        assert torch.equal(y[others], want[0][others]) and torch.equal(lse[others], want[1][others]), bad
        for row, head in hit:
            assert y[row, head].isnan().all() and lse[row, head].isnan(), (bad, row, head)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("counts", [[1, 1, 1], [3, 4, 2], [50, 60, 40]])
def test_nan_in_rows_that_see_nothing(q4lib, gpu, dtype, counts):
    """They have y 0 and lse -infinity as any such row: no positions, or no page for any."""
    b = Batch([0, 70, 90], counts, 16, single=counts[0] == 1)
    b.tables[1] = -1
    cache, q = random_cache(1, b.pages, 2, 16, 64), rows(2, dtype, b.tokens, 4, 64)
    q[::2, :, 7], q[1::2, :, 9] = math.nan, math.inf
    for kw in (dict(), dict(scale=0.0), dict(softcap=5.0)):
        y, lse = q4lib.q4_attention(q.to(gpu), torch.from_numpy(cache).to(gpu), *b.device(gpu), return_lse=True, **kw)
        n = counts[0] + counts[1]
        assert (y[:n] == 0).all() and (lse[:n] == -math.inf).all()
        assert y[n:].isnan().all() and lse[n:].isnan().all()


# ------------------------------------------------------------------ strides

@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_one_row_of_rows_that_are_no_whole_pieces_apart(q4lib, gpu, dtype):
    """The first of rows that lie an odd number of elements apart: a row alone has no stride."""
    b = Batch([37], [1], 16, single=True)
    cache = torch.from_numpy(random_cache(1, b.pages, 2, 16, 64)).to(gpu)
    tables, lengths, _ = b.device(gpu)
    wide = rows(2, dtype, 3, 8 * 64 + 1).to(gpu)
    qkv = wide.as_strided((1, 8, 64), (8 * 64 + 1, 64, 1))
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    assert q.stride(0) == 8 * 64 + 1
    one, two = cache.clone(), cache.clone()
    q4lib.q4_cache_write(k.contiguous(), v.contiguous(), one, tables, lengths)
    want = q4lib.q4_attention(q.contiguous(), one, tables, lengths)
    q4lib.q4_cache_write(k, v, two, tables, lengths)
    assert torch.equal(one, two)
    assert torch.equal(q4lib.q4_attention(q, two, tables, lengths), want)
    y = torch.empty_like(want)
    assert torch.equal(q4lib.q4_attention(q, two, tables, lengths, y=y), want)
    fast = q4lib._fast()
    assert fast.cache_write(k, v, two, tables, lengths, None) is True
    assert torch.equal(fast.attention(q, two, tables, lengths, None, None, True, 0, 0.0, False), want)


# ------------------------------------------------------------------ numbers of rows

@pytest.mark.parametrize("with_offsets", [False, True])
@pytest.mark.parametrize("tokens", [-1, 0, 1 << 63, 1 << 70])
def test_numbers_of_rows_that_are_none(q4lib, gpu, tokens, with_offsets):
    """Reading back refuses them (-1 was taken for one row a sequence)."""
    b = Batch([37, 5], [1, 1], 16)
    cache = q4lib.q4_cache(b.pages, 16, 2, 64, device=gpu)
    tables, lengths, offsets = b.device(gpu)
    with pytest.raises((ValueError, RuntimeError, TypeError)):
        q4lib.q4_cache_read(cache, tables, lengths, offsets if with_offsets else None, tokens=tokens)
    k, _ = q4lib.q4_cache_read(cache, tables, lengths)
    assert k.shape == (2, 2, 64)


# ------------------------------------------------------------------ what is rounded

@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("name", FEW)
@pytest.mark.parametrize("kw", [dict(), dict(window=3), dict(softcap=2.0), dict(scale=-0.5)])
def test_few_rows_round_neither_keys_nor_weights_of_fp16_q(q4lib, gpu, dtype, name, kw):
    """Keys' codes and scales as they are, weights of fp16 q in two parts: held to bounds that
    a key rounded to fp16, or a weight in one part, leaves."""
    b, cache, q = few_example(name, dtype)
    same(q4lib, gpu, b, cache, q, f"{dtype} {name} {kw}", y_dtype=torch.float32, **kw)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("name", WAYS)
@pytest.mark.parametrize("kw", [dict(), dict(window=70), dict(causal=False), dict(scale=-0.3)])
def test_every_way_within_what_it_rounds(q4lib, gpu, dtype, name, kw):
    b, cache, q = example(name, dtype)
    same(q4lib, gpu, b, cache, q, f"{dtype} {name} {kw}", y_dtype=torch.float32, **kw)


# ------------------------------------------------------------------ positions that are not split

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,heads", [(32, 400), (64, 400), (96, 160), (128, 160), (160, 80), (192, 80), (224, 80),
                                     (256, 80)])
@pytest.mark.parametrize("empty", [0, 40])
def test_prompts_of_as_many_workgroups_as_there_is_room_for(q4lib, gpu, dtype, d, heads, empty):
    """Rows leave the workgroup that has all their positions (with fewer workgroups the positions are
    split and the rows joined by another launch); alone, and where the batch's rows are few on
    average."""
    n = 500
    b = Batch([n + 30] + [3] * empty, [n] + [0] * empty, 64, seed=d)
    assert (n + 127) // 128 * heads >= 256 * (1 if d > 128 else 2 if d > 64 else 3)
    cache, q = random_cache(1, b.pages, heads, 64, d), rows(2, dtype, b.tokens, heads, d)
    same(q4lib, gpu, b, cache, q, f"{dtype} {heads} x {d}")
