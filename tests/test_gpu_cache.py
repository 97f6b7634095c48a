"""The paged cache: bytes written and values read, against the oracle's quantiser and
the layout that the public header states, byte by byte."""

import math

import numpy as np
import pytest
import torch

from _cache import TYPES, Batch, decoded, random_cache, rows, written

pytestmark = pytest.mark.gpu

# lengths, rows, page size: one position; granules cut at both ends; pages that end
# inside a granule run; no rows; no positions; more rows than positions
SHAPES = [
    ([1], [1], 16), ([17], [1], 16), ([16], [16], 16), ([33], [33], 32), ([100], [37], 16),
    ([5, 0, 48, 31], [5, 0, 17, 31], 16), ([3, 130, 64], [7, 2, 64], 64), ([1000, 999], [130, 1], 48),
    ([40] * 70, [1, 2, 3, 0, 17] * 14, 16)]


def values_of(cache, batch, kv, d, dtype, value):
    out = torch.full((batch.tokens, kv, d), math.nan, dtype=torch.float64)
    for row, s, t in batch.places:
        x = decoded(cache, batch, s, t, value) if 0 <= t < batch.lengths[s] else None
        out[row] = torch.zeros(kv, d) if x is None else torch.from_numpy(x)
    return out


def same(got, want, dtype):
    """Rounded once; rows of no sequence (NaN) are not compared."""
    w = want.to(TYPES[dtype]).double()
    ok = want.isnan() | (got.cpu().double() == w)
    assert ok.all(), (int((~ok).sum()), (~ok).nonzero()[0])


@pytest.mark.parametrize("lengths,counts,page", SHAPES)
@pytest.mark.parametrize("dtype,kv,d", [("f16", 2, 128), ("bf16", 1, 32), ("f32", 3, 96), ("f16", 1, 256),
                                        ("bf16", 5, 64)])
def test_bytes_written_and_values_read(q4lib, gpu, lengths, counts, page, dtype, kv, d):
    b = Batch(lengths, counts, page, seed=len(lengths) + d, before=2, behind=3)
    k, v = rows(1, dtype, b.tokens, kv, d, scale=2.0), rows(2, dtype, b.tokens, kv, d, scale=0.1)
    old = random_cache(3, b.pages, kv, page, d)
    cache = torch.from_numpy(old).to(gpu)
    tables, ls, offsets = b.device(gpu)
    q4lib.q4_cache_write(k.to(gpu), v.to(gpu), cache, tables, ls, offsets)
    want = written(old, b, k, v)
    assert np.array_equal(cache.cpu().numpy(), want)  # (every byte that is not a row's is as it was)
    for out in ("f32", "f16", "bf16"):
        kg = torch.full((b.tokens, kv, d), 7.0, dtype=TYPES[out], device=gpu)
        vg = kg.clone()
        q4lib.q4_cache_read(cache, tables, ls, offsets, k=kg, v=vg)
        same(kg, values_of(want, b, kv, d, out, 0), out)
        same(vg, values_of(want, b, kv, d, out, 1), out)
        outside = [0, 1] + list(range(b.tokens - 3, b.tokens))
        assert (kg[outside] == 7).all() and (vg[outside] == 7).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_one_row_each_without_offsets(q4lib, gpu, dtype):
    """As with offsets 0, 1, 2, ..; a sequence without positions stores nothing and reads zeros."""
    lengths = [1, 16, 17, 0, 300, 64]
    b = Batch(lengths, [1] * 6, 16, single=True)
    kv, d = 2, 128
    k, v = rows(1, dtype, 6, kv, d), rows(2, dtype, 6, kv, d)
    old = random_cache(3, b.pages, kv, 16, d)
    cache = torch.from_numpy(old).to(gpu)
    tables, ls, _ = b.device(gpu)
    q4lib.q4_cache_write(k.to(gpu), v.to(gpu), cache, tables, ls)
    want = written(old, b, k, v)
    assert np.array_equal(cache.cpu().numpy(), want)
    kg, vg = q4lib.q4_cache_read(cache, tables, ls, dtype=TYPES[dtype])
    same(kg, values_of(want, b, kv, d, dtype, 0), dtype)
    same(vg, values_of(want, b, kv, d, dtype, 1), dtype)
    assert (kg[3] == 0).all() and (vg[3] == 0).all()


def test_rows_of_a_fused_product(q4lib, gpu):
    """k and v where a q/k/v product leaves them, and pages of 16 to 512 positions."""
    kv, heads, d = 2, 6, 64
    for page in (16, 32, 48, 512):
        b = Batch([70, 20], [70, 9], page)
        qkv = rows(5, "bf16", b.tokens, heads + 2 * kv, d)
        old = random_cache(3, b.pages, kv, page, d)
        cache = torch.from_numpy(old).to(gpu)
        dev = qkv.to(gpu)
        q4lib.q4_cache_write(dev[:, heads:heads + kv], dev[:, heads + kv:], cache, *b.device(gpu))
        assert np.array_equal(cache.cpu().numpy(), written(old, b, qkv[:, heads:heads + kv], qkv[:, heads + kv:]))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_extreme_values_are_limited(q4lib, gpu, dtype):
    """Infinities, NaN, the type's largest and smallest values, zeros, one block of each."""
    kv, d = 1, 256
    x = rows(5, dtype, 16, kv, d)
    big = torch.finfo(TYPES[dtype]).max
    for i, v in enumerate((math.inf, -math.inf, math.nan, big, -big, 65504.0, 0.0, -0.0,
                           torch.finfo(TYPES[dtype]).tiny)):
        x[i, 0, 32:64] = v
        x[i, 0, 70] = v
    x[9, 0, :32] = torch.tensor([math.inf, -math.inf] * 16)
    x[10] = math.nan
    b = Batch([16], [16], 16)
    old = random_cache(3, b.pages, kv, 16, d)
    cache = torch.from_numpy(old).to(gpu)
    q4lib.q4_cache_write(x.to(gpu), x.flip(0).contiguous().to(gpu), cache, *b.device(gpu))
    want = written(old, b, x, x.flip(0))
    assert np.array_equal(cache.cpu().numpy(), want)
    k, v = q4lib.q4_cache_read(cache, *b.device(gpu), tokens=16, dtype=torch.float32)
    assert torch.isfinite(k).all() and torch.isfinite(v).all()


def test_pages_that_are_none(q4lib, gpu):
    """Page numbers outside the cache: not written, read as zeros; lengths beyond the tables are cut."""
    kv, d, page = 2, 64, 16
    b = Batch([90, 64], [90, 64], page)
    b.tables[0, 1], b.tables[0, 3], b.tables[1, 0] = -5, b.pages, 2 ** 31 - 1
    k, v = rows(1, "f16", b.tokens, kv, d), rows(2, "f16", b.tokens, kv, d)
    old = random_cache(3, b.pages, kv, page, d)
    cache = torch.from_numpy(old).to(gpu)
    q4lib.q4_cache_write(k.to(gpu), v.to(gpu), cache, *b.device(gpu))
    want = written(old, b, k, v)
    assert np.array_equal(cache.cpu().numpy(), want)
    kg, vg = q4lib.q4_cache_read(cache, *b.device(gpu), tokens=b.tokens)
    same(kg, values_of(want, b, kv, d, "f16", 0), "f16")
    same(vg, values_of(want, b, kv, d, "f16", 1), "f16")
    # 4 tables of 16 positions hold 64; rows of a length of 80 are its last
    c = Batch([64], [20], page)
    tables, _, offsets = c.device(gpu)
    cache = torch.from_numpy(old).to(gpu)
    far = torch.tensor([80], dtype=torch.int32, device=gpu)
    q4lib.q4_cache_write(k[:20].to(gpu), v[:20].to(gpu), cache, tables, far, offsets)
    assert np.array_equal(cache.cpu().numpy(), written(old, c, k[:20], v[:20]))


def test_offsets_that_make_no_sense(q4lib, gpu):
    """Falling and far offsets, negative lengths: no access outside, other sequences as they are."""
    kv, d = 1, 64
    k = rows(1, "f16", 12, kv, d).to(gpu)
    tables = torch.zeros((3, 2), dtype=torch.int32, device=gpu)
    for offsets, lengths in (([5, 2, -9, 4], [20, 20, 20]), ([0, 4, 1 << 30, 1 << 30], [30, -3, 1 << 30]),
                             ([-7, -7, -7, 12], [32, 32, 32])):
        cache = q4lib.q4_cache(1, 16, kv, d, device=gpu)
        args = (cache, tables, torch.tensor(lengths, dtype=torch.int32, device=gpu),
                torch.tensor(offsets, dtype=torch.int32, device=gpu))
        q4lib.q4_cache_write(k, k, *args)
        out = q4lib.q4_cache_read(*args, tokens=12)
        torch.cuda.synchronize()
        assert out[0].shape == (12, kv, d)


def test_a_cache_of_more_than_4_gib(q4lib, gpu):
    """Pages on both sides of 2^32 bytes."""
    kv, d, page = 8, 128, 64
    pages = (1 << 32) // (kv * 2 * 4 * 9 * d) + 3
    cache = torch.zeros((pages, kv, 2, page // 16, 9 * d), dtype=torch.uint8, device=gpu)
    assert cache.numel() > 1 << 32
    x = rows(1, "f16", 200, kv, d).to(gpu)
    y = rows(2, "f16", 200, kv, d).to(gpu)
    ids = torch.tensor([[pages - 1, 0, pages - 2, 1]], dtype=torch.int32, device=gpu)
    ls, offs = torch.tensor([200], dtype=torch.int32, device=gpu), torch.tensor([0, 200], dtype=torch.int32, device=gpu)
    q4lib.q4_cache_write(x, y, cache, ids, ls, offs)
    small = q4lib.q4_cache(4, page, kv, d, device=gpu)
    near = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32, device=gpu)
    q4lib.q4_cache_write(x, y, small, near, ls, offs)
    assert torch.equal(cache[[0, 1, pages - 2, pages - 1]], small)
    for a, b in zip(q4lib.q4_cache_read(cache, ids, ls, offs, tokens=200),
                    q4lib.q4_cache_read(small, near, ls, offs, tokens=200)):
        assert torch.equal(a, b)
