"""Attention over the paged Q4_0 cache against its formula in 64 bits."""

import math

import pytest
import torch

from _cache import TYPES, Batch, attention64, check, random_cache, rows

pytestmark = pytest.mark.gpu


def run(q4lib, gpu, b, dtype, heads, kv, d, seed=1, qscale=1.0, few=None, y_dtype=None, cache_scale=1.0, **kw):
    cache = random_cache(seed, b.pages, kv, b.page, d, scale=cache_scale)
    q = rows(seed + 1, dtype, b.tokens, heads, d, scale=qscale)
    y = torch.full((b.tokens, heads, d), 7.0, dtype=TYPES[y_dtype or dtype], device=gpu)
    lse = torch.full((b.tokens, heads), 7.0, device=gpu)
    out = q4lib.q4_attention(q.to(gpu), torch.from_numpy(cache).to(gpu), *b.device(gpu), return_lse=True, y=y,
                             lse=lse, **kw)
    assert out[0] is y and out[1] is lse
    want, bound, big, lbound = attention64(q, cache, b, dtype=y.dtype, **kw)
    what = f"{dtype} {heads}/{kv} x {d} {b.lengths[:4]} {b.counts[:4]} page {b.page} {kw}"
    check(y, want, bound, what)
    check(lse, big, lbound, "lse " + what)
    free = want.isnan()
    assert (y.cpu()[free] == 7).all() and (lse.cpu()[big.isnan()] == 7).all()
    return y


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("heads,kv", [(5, 1), (4, 4), (16, 1), (40, 2)])
def test_one_token(q4lib, gpu, dtype, d, heads, kv):
    """Lengths around granules and tiles, none at all, and some thousands."""
    b = Batch([1, 15, 16, 17, 63, 64, 65, 0, 130, 1000, 2085], [1] * 11, 16, single=True)
    run(q4lib, gpu, b, dtype, heads, kv, d)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("page", [16, 32, 48, 128, 1024])
@pytest.mark.parametrize("kw", [{}, dict(window=1), dict(window=50), dict(window=300, softcap=3.0),
                                dict(causal=False), dict(causal=False, window=20), dict(scale=-0.3), dict(scale=0.0)])
def test_few_rows(q4lib, gpu, dtype, page, kw):
    """Drafts of several tokens, sequences without rows and with more rows than positions,
    rows before the first and behind the last sequence."""
    b = Batch([40, 200, 3, 70, 0, 513], [3, 6, 5, 0, 2, 4], page, seed=page, before=1, behind=2)
    run(q4lib, gpu, b, dtype, 10, 2, 64, **kw)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("d,heads,kv", [(128, 10, 2), (64, 3, 3), (96, 8, 1), (256, 4, 2), (32, 2, 1), (192, 6, 2)])
@pytest.mark.parametrize("kw", [{}, dict(window=70), dict(softcap=5.0), dict(causal=False), dict(scale=-0.2, window=40), dict(scale=0.0)])
def test_many_rows(q4lib, gpu, dtype, d, heads, kv, kw):
    """Prompts, a chunk behind a history, and single tokens among them."""
    b = Batch([130, 61, 400, 300], [130, 61, 90, 1], 32, seed=d, before=2, behind=1)
    run(q4lib, gpu, b, dtype, heads, kv, d, **kw)


@pytest.mark.parametrize("dtype,y_dtype", [("f16", "f32"), ("bf16", "f32"), ("f32", "bf16"), ("bf16", "f16")])
def test_output_types(q4lib, gpu, dtype, y_dtype):
    run(q4lib, gpu, Batch([100, 300], [1, 1], 16, single=True), dtype, 8, 2, 128, y_dtype=y_dtype)
    run(q4lib, gpu, Batch([100, 300], [100, 70], 16), dtype, 8, 2, 128, y_dtype=y_dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("counts", [[1, 1], [90, 40]])
def test_sharp_and_flat_softmax(q4lib, gpu, dtype, counts):
    """Scores of hundreds, where one weight is all; of nothing, where all are alike."""
    for qscale, cs in ((40.0, 1.0), (1e-6, 1.0), (1.0, 60.0)):
        run(q4lib, gpu, Batch([700, 333], counts, 64), dtype, 8, 2, 128, qscale=qscale, cache_scale=cs)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("heads", [33, 64, 100])
def test_many_heads_of_one_kv_head(q4lib, gpu, dtype, heads):
    run(q4lib, gpu, Batch([100, 257], [1, 1], 16, single=True), dtype, heads, 1, 64)
    run(q4lib, gpu, Batch([100, 257], [3, 40], 16), dtype, heads, 1, 64)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("counts", [[1, 1], [2, 5], [120, 200]])
def test_unseen_places_may_hold_anything(q4lib, gpu, dtype, counts):
    """NaN and infinite scales behind the last position and in pages that no table names; a
    page number that names no page inside a sequence."""
    import numpy as np
    b = Batch([200, 333], counts, 48, spare=3)
    b.tables[1, 2] = b.pages + 7
    kv, d, heads = 2, 128, 6
    cache = random_cache(1, b.pages, kv, 48, d)
    live = np.zeros((b.pages, 48), dtype=bool)
    for s in range(2):
        for t in range(b.lengths[s]):
            if b.page_of(s, t) >= 0:
                live[b.page_of(s, t), t % 48] = True
    halves = cache.view(np.uint16)  # [.., 9 d / 2]
    for p, t in zip(*np.nonzero(~live)):
        from _cache import index
        for value in (0, 1):
            _, at = index(d, value, t % 16)
            halves[p, :, value, t // 16][:, at // 2] = 0x7E00 if t % 2 else 0xFC00
    q = rows(2, dtype, b.tokens, heads, d)
    for kw in ({}, dict(causal=False), dict(window=30)):
        y, lse = q4lib.q4_attention(q.to(gpu), torch.from_numpy(cache).to(gpu), *b.device(gpu), return_lse=True, **kw)
        want, bound, big, lbound = attention64(q, cache, b, **kw)
        check(y, want, bound, str(kw))
        check(lse, big, lbound, str(kw))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_a_sequence_without_any_page(q4lib, gpu, dtype):
    b = Batch([70, 40, 50], [1, 30, 2], 16)
    b.tables[1] = -1
    b.tables[2, 0] = 1 << 30
    run(q4lib, gpu, b, dtype, 4, 2, 64)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_rows_of_a_fused_product(q4lib, gpu, dtype):
    """q where a q/k/v product leaves it: the same bits as a copy."""
    heads, kv, d = 6, 2, 128
    for counts in ([1, 1, 1], [50, 3, 70]):
        b = Batch([100, 64, 200], counts, 16)
        cache = torch.from_numpy(random_cache(1, b.pages, kv, 16, d)).to(gpu)
        qkv = rows(3, dtype, b.tokens, heads + 2 * kv, d).to(gpu)
        a = q4lib.q4_attention(qkv[:, :heads], cache, *b.device(gpu))
        assert torch.equal(a, q4lib.q4_attention(qkv[:, :heads].contiguous(), cache, *b.device(gpu)))
        assert math.isfinite(float(a.float().abs().max()))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_long_history(q4lib, gpu, dtype):
    """One token over some ten thousand positions, and a batch of very unequal lengths."""
    run(q4lib, gpu, Batch([20011], [1], 256, single=True), dtype, 10, 2, 128)
    run(q4lib, gpu, Batch([9000, 1, 5, 700, 64, 129], [1] * 6, 16, single=True), dtype, 5, 1, 64)
    run(q4lib, gpu, Batch([9000, 40, 5], [2, 1, 3], 16), dtype, 5, 1, 64, window=8000)
