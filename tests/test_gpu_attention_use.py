"""The paged Q4_0 cache and the attention over it as they are used: a decoder layer's
attention from its products on, captured and replayed decode steps, two streams, caches
of more than 4 GiB, prefixes that sequences share, thousands of sequences."""

import math

import numpy as np
import pytest
import torch

from _cache import TYPES, Batch, attention64, check, random_cache, rows, written
from _fused import weights

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.uint8)


class Layer:
    """Attention of a decoder layer: q/k/v product, cache, attention, product of its output."""

    def __init__(self, gpu, hidden, heads, kv, d, dtype, seed=1):
        self.heads, self.kv, self.d, self.dtype = heads, kv, d, dtype
        self.qkv = weights(seed, 1, (heads + 2 * kv) * d, hidden)[0][0].to(gpu)
        self.out = weights(seed + 1, 1, hidden, heads * d)[0][0].to(gpu)

    def parts(self, q4, x):
        qkv = q4.q4_linear(x, self.qkv).unflatten(1, (self.heads + 2 * self.kv, self.d))
        return qkv[:, :self.heads], qkv[:, self.heads:self.heads + self.kv], qkv[:, self.heads + self.kv:]

    def run(self, q4, x, cache, tables, lengths, offsets=None, **kw):
        q, k, v = self.parts(q4, x)
        q4.q4_cache_write(k, v, cache, tables, lengths, offsets)
        y = q4.q4_attention(q, cache, tables, lengths, offsets, **kw)
        return q4.q4_linear(y.flatten(1), self.out, residual=x)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("heads,kv,d,page", [(8, 2, 64, 16), (3, 3, 128, 48), (6, 1, 96, 256)])
def test_prompts_then_tokens(q4lib, gpu, dtype, heads, kv, d, page):
    """Prompts, a chunk and drafts at once, then single tokens: after each step the cache's
    bytes are those of the keys and values written so far, and the attention's rows the
    formula's over them."""
    hidden = 320
    L = Layer(gpu, hidden, heads, kv, d, dtype)
    lengths, counts = [70, 3, 130, 33], [70, 3, 130, 33]
    room = Batch([n + 20 for n in lengths], [0] * 4, page, seed=d)  # pages for what is to come
    cache = q4lib.q4_cache(room.pages, page, kv, d, device=gpu)
    host = cache.cpu().numpy()
    for step in range(5):
        b = Batch(lengths, counts, page, single=step > 2)
        b.tables, b.max_pages, b.pages = room.tables, room.max_pages, room.pages
        x = rows(20 + step, dtype, b.tokens, hidden).to(gpu)
        tables, lens, offsets = b.device(gpu)
        q, k, v = L.parts(q4lib, x)
        y = L.run(q4lib, x, cache, tables, lens, offsets)
        host = written(host, b, k.cpu(), v.cpu())
        assert np.array_equal(cache.cpu().numpy(), host), step
        a = q4lib.q4_attention(q, cache, tables, lens, offsets)
        want, bound, _, _ = attention64(q.cpu(), host, b)
        check(a, want, bound, f"step {step}")
        assert torch.equal(y, q4lib.q4_linear(a.flatten(1), L.out, residual=x))
        counts = [[4, 0, 7, 1], [1, 2, 0, 3], [1] * 4, [1] * 4][min(step, 3)]
        lengths = [n + c for n, c in zip(lengths, counts)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("start,page", [([5, 700, 1, 64], 16), ([30, 100, 2, 15], 32), ([1200, 3000, 1, 64], 16)])
def test_captured_steps(q4lib, gpu, dtype, start, page):
    """A decode step of a layer in a graph that counts its lengths on: every replay, with the
    program's own work between, leaves the bits of the same steps run eagerly.  Two graphs
    by turns, each with its cache."""
    hidden, heads, kv, d = 256, 8, 2, 64
    L = Layer(gpu, hidden, heads, kv, d, dtype)
    room = Batch([n + 16 for n in start], [1] * 4, page, single=True)
    tables = torch.from_numpy(room.tables).to(gpu)
    first = torch.from_numpy(random_cache(3, room.pages, kv, page, d)).to(gpu)
    steps = [rows(40 + i, dtype, 4, hidden).to(gpu) for i in range(5)]
    cache, lens, want = first.clone(), torch.tensor(start, dtype=torch.int32, device=gpu), []
    for x in steps:
        lens += 1
        want.append((L.run(q4lib, x, cache, tables, lens), cache.clone()))
    graphs = []
    for _ in range(2):
        x, cache = steps[0].clone(), first.clone()
        lens = torch.tensor(start, dtype=torch.int32, device=gpu)
        warm = lens + 1
        L.run(q4lib, x, first.clone(), tables, warm)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lens += 1
            y = L.run(q4lib, x, cache, tables, lens)
        graphs.append((g, x, y, cache, lens))  # (what a graph reads and writes lives as long)
    for i, step in enumerate(steps):
        for g, x, y, cache, _ in graphs:
            x.copy_(step)
            g.replay()
            junk = torch.randn(256, 256, device=gpu) @ torch.randn(256, 256, device=gpu)  # noqa: F841
            L.run(q4lib, steps[0], first.clone(), tables, warm)
            torch.cuda.synchronize()
        for g, x, y, cache, _ in graphs:
            assert torch.equal(bits(y), bits(want[i][0])), i
            assert torch.equal(cache, want[i][1]), i


def test_captured_mixed_batch(q4lib, gpu):
    """A batch whose offsets and lengths change between replays: prompts, drafts, padding."""
    kv, heads, d, page, tokens, seqs = 2, 6, 128, 16, 200, 5
    tables = torch.arange(seqs * 40, dtype=torch.int32, device=gpu).view(seqs, 40).flip(0).contiguous()
    cache = torch.from_numpy(random_cache(5, seqs * 40, kv, page, d)).to(gpu)
    q = rows(6, "bf16", tokens, heads, d).to(gpu)
    lens = torch.zeros(seqs, dtype=torch.int32, device=gpu)
    offsets = torch.zeros(seqs + 1, dtype=torch.int32, device=gpu)
    y = torch.zeros(tokens, heads, d, dtype=torch.bfloat16, device=gpu)
    q4lib.q4_attention(q, cache, tables, lens, offsets, y=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q4lib.q4_attention(q, cache, tables, lens, offsets, y=y)
    for counts, lengths in (([200, 0, 0, 0, 0], [640, 1, 0, 5, 6]), ([1, 1, 1, 1, 1], [640, 600, 17, 1, 300]),
                            ([50, 1, 100, 4, 0], [50, 640, 100, 333, 0]), ([0, 0, 0, 0, 0], [9, 9, 9, 9, 9]),
                            ([11, 10, 12, 0, 60], [500, 10, 5, 0, 60])):
        offsets.copy_(torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).int())
        lens.copy_(torch.tensor(lengths, dtype=torch.int32))
        y.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        want = torch.full_like(y, 3.0)
        q4lib.q4_attention(q, cache, tables, lens, offsets, y=want)
        assert torch.equal(bits(y), bits(want)), counts
        assert (y[sum(counts):] == 3).all()


BATCHES = {
    "wide": (Batch([5000, 700], [1, 1], 16, single=True), 8, 2, 128),
    "heads": (Batch([600 + 50 * i for i in range(30)], [1] * 30, 32, seed=1, single=True), 8, 4, 64),
    "cut": (Batch([(37 * i) % 800 for i in range(300)], [1] * 300, 64, seed=2, single=True), 4, 2, 32),
    "whole": (Batch([100, 400, 7], [1, 1, 1], 16, seed=3, single=True), 4, 2, 128),
    "drafts": (Batch([900, 1300, 40], [5, 2, 3], 16, seed=4), 10, 2, 128),
    "mixed": (Batch([900, 700, 300], [1, 150, 300], 16, seed=5, before=1, behind=3), 4, 1, 96),
    "prompts": (Batch([1500, 400], [1500, 400], 128, seed=6), 4, 4, 256),
    "row": (Batch([30, 600], [30, 2], 16, seed=7), 4, 2, 64),
}


def example(name, gpu, dtype, seed=9):
    b, heads, kv, d = BATCHES[name]
    cache = random_cache(seed, b.pages, kv, b.page, d)
    q = rows(seed + 1, dtype, b.tokens, heads, d)
    return b, cache, q, [q.to(gpu), torch.from_numpy(cache).to(gpu)] + b.device(gpu)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("name", BATCHES)
@pytest.mark.parametrize("kw", [{}, dict(window=600, softcap=20.0)])
def test_ways_of_cutting_the_work(q4lib, gpu, dtype, name, kw):
    """Batches that are cut and joined in each of the ways there are; the caller's workspace,
    of any contents; the short way from Python and the full one; twice: the same bits."""
    b, cache, q, args = example(name, gpu, dtype)
    y, lse = q4lib.q4_attention(*args, return_lse=True, **kw)
    want, bound, big, lbound = attention64(q, cache, b, **kw)
    check(y, want, bound, name)
    check(lse, big, lbound, "lse " + name)
    mine = ~want.isnan().to(gpu)
    code = {"f32": 0, "f16": 1, "bf16": 2}[dtype]
    need = q4lib.q4_attention_workspace_size(b.seqs, b.tokens, q.shape[1], cache.shape[1], q.shape[2], code,
                                             b.offsets is not None)
    for fill in (0, 0xFF, 0x7C, 0x01):
        ws = torch.full((max(need, 1),), fill, dtype=torch.uint8, device=gpu)
        z = torch.empty_like(y)
        zl = torch.empty_like(lse)
        out = q4lib.q4_attention(*args, y=z, lse=zl, return_lse=True, workspace=ws, **kw)
        assert out[0] is z and torch.equal(z[mine], y[mine]), hex(fill)
        assert torch.equal(zl[mine[..., 0]], lse[mine[..., 0]])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_two_streams(q4lib, gpu, dtype):
    """Calls of every kind on two streams at once, given as argument and as the current one."""
    work = [example(name, gpu, dtype) for name in BATCHES]
    want = [q4lib.q4_attention(*args) for *_, args in work]
    mine = [~attention64(q, cache, b)[0].isnan().to(gpu) for b, cache, q, _ in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for turn in range(3):
        for i, (*_, args) in enumerate(work):
            got[0].append(q4lib.q4_attention(*args, stream=streams[0]))
            with torch.cuda.stream(streams[1]):
                got[1].append(q4lib.q4_attention(*work[-1 - i][-1]))
    torch.cuda.synchronize()
    n = len(work)
    for j in range(3 * n):
        assert torch.equal(got[0][j][mine[j % n]], want[j % n][mine[j % n]]), j
        k = n - 1 - j % n
        assert torch.equal(got[1][j][mine[k]], want[k][mine[k]]), j


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("counts", [[1, 1, 1], [3, 50, 100]])
def test_sequences_that_share_pages(q4lib, gpu, dtype, counts):
    """A common prefix's pages in several tables, and a page twice in one table."""
    b = Batch([300, 300, 200], counts, 32, seed=8, single=counts == [1, 1, 1])
    b.tables[1, :5] = b.tables[0, :5]
    b.tables[2, :3] = b.tables[0, :3]
    b.tables[2, 3] = b.tables[2, 1]
    cache = random_cache(2, b.pages, 2, 32, 128)
    q = rows(3, dtype, b.tokens, 6, 128)
    y = q4lib.q4_attention(q.to(gpu), torch.from_numpy(cache).to(gpu), *b.device(gpu))
    want, bound, _, _ = attention64(q, cache, b)
    check(y, want, bound)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_cache_of_more_than_4_gib(q4lib, gpu, dtype):
    """Pages on either side of 2^31 and 2^32 bytes, for few rows and for many."""
    kv, d, page = 2, 128, 64
    size = kv * 2 * page // 16 * 9 * d
    pages = (2 ** 32 + 2 ** 29) // size
    big = torch.empty((pages, kv, 2, page // 16, 9 * d), dtype=torch.uint8, device=gpu)
    for counts in ([1, 1], [70, 3]):
        b = Batch([290, 200], counts, page, seed=1, spare=0, single=counts == [1, 1])
        at = [0, 1, 2 ** 31 // size - 1, 2 ** 31 // size, 2 ** 31 // size + 1, 2 ** 32 // size - 1, 2 ** 32 // size,
              2 ** 32 // size + 1, pages - 1]
        assert b.pages == len(at)
        cache = random_cache(4, b.pages, kv, page, d)
        for i, p in enumerate(at):
            big[p] = torch.from_numpy(cache[i]).to(gpu)
        tables, lens, offsets = b.device(gpu)
        far = torch.tensor(at, dtype=torch.int32, device=gpu)
        tables = torch.where(tables >= 0, far[tables.clamp(min=0).long()], tables)
        q = rows(5, dtype, b.tokens, 4, d)
        y = q4lib.q4_attention(q.to(gpu), big, tables, lens, offsets)
        want, bound, _, _ = attention64(q, cache, b)
        check(y, want, bound, str(counts))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("single", [True, False])
def test_thousands_of_sequences(q4lib, gpu, dtype, single):
    """More sequences than a workgroup has lanes, many of them empty; every fifth has no rows
    and one has many."""
    seqs = 2600
    rng = np.random.default_rng(3)
    lengths = [int(n) for n in rng.integers(0, 40, seqs)]
    counts = [1] * seqs if single else [0 if s % 5 == 0 else 1 + s % 3 for s in range(seqs)]
    if not single:
        lengths[1300], counts[1300] = 150, 150
    b = Batch(lengths, counts, 16, seed=4, single=single)
    cache = random_cache(5, b.pages, 1, 16, 32)
    q = rows(6, dtype, b.tokens, 2, 32)
    y, lse = q4lib.q4_attention(q.to(gpu), torch.from_numpy(cache).to(gpu), *b.device(gpu), return_lse=True)
    want, bound, big, lbound = attention64(q, cache, b)
    check(y, want, bound)
    check(lse, big, lbound)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_heads_by_the_thousand(q4lib, gpu, dtype):
    """One kv head for a thousand heads; a thousand kv heads."""
    for heads, kv in ((1000, 1), (1000, 1000)):
        for b in (Batch([70, 600], [1, 1], 16, single=True), Batch([70, 33], [2, 33], 16)):
            cache = random_cache(5, b.pages, kv, 16, 32)
            q = rows(6, dtype, b.tokens, heads, 32)
            y = q4lib.q4_attention(q.to(gpu), torch.from_numpy(cache).to(gpu), *b.device(gpu))
            want, bound, _, _ = attention64(q, cache, b)
            check(y, want, bound, str((heads, kv)))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_batches_that_make_no_sense(q4lib, gpu, dtype):
    """Lengths below zero and beyond the tables, offsets that fall or leave the rows: rows are
    written where the offsets, limited to the rows, say, and nothing else is touched."""
    kv, heads, d, page = 1, 2, 64, 16
    cache = random_cache(1, 8, kv, page, d)
    tables = torch.arange(8, dtype=torch.int32).view(2, 4)
    q = rows(2, dtype, 6, heads, d)
    for lengths, offsets in (([-5, 1000], [0, 2, 6]), ([2 ** 31 - 1, -2 ** 31], [0, 3, 2 ** 31 - 1]),
                             ([64, 30], [5, 2, 4]), ([64, 64], [-7, 3, 3])):
        y = torch.full((6, heads, d), 9.0, dtype=TYPES[dtype], device=gpu)
        lens = torch.tensor(lengths, dtype=torch.int64).to(torch.int32)
        q4lib.q4_attention(q.to(gpu), torch.from_numpy(cache).to(gpu), tables.to(gpu), lens.to(gpu),
                           torch.tensor(offsets, dtype=torch.int32, device=gpu), y=y)
        free = torch.ones(6, dtype=torch.bool)
        for s in range(2):
            lo, hi = min(max(offsets[s], 0), 6), min(max(offsets[s + 1], 0), 6)
            if hi > lo:
                free[lo:hi] = False
                b = Batch([min(max(lengths[s], 0), 64)], [hi - lo], page)
                b.tables, b.pages, b.max_pages = tables[s:s + 1].numpy(), 8, 4
                want, bound, _, _ = attention64(q[lo:hi], cache, b)
                check(y[lo:hi], want, bound, str((lengths, offsets, s)))
        assert (y.cpu()[free] == 9).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("name", BATCHES)
def test_rows_that_are_no_numbers(q4lib, gpu, dtype, name):
    """NaN or an infinity in a row and head of q: that one has no number in y and lse, every other one
    the same bits."""
    b, cache, q, args = example(name, gpu, dtype)
    want = q4lib.q4_attention(*args)
    row, head = b.places[len(b.places) // 2][0], q.shape[1] // 2
    for bad in (math.nan, math.inf, -math.inf):
        x = args[0].clone()
        x[row, head, 3] = bad
        y, lse = q4lib.q4_attention(x, *args[1:], return_lse=True)
        others = torch.zeros(b.tokens, q.shape[1], dtype=torch.bool, device=gpu)
        for r, *_ in b.places:
            others[r] = True
        others[row, head] = False
        assert torch.equal(y[others], want[others]), bad
        if math.isnan(bad) and b.lengths[b.places[len(b.places) // 2][1]] > 0:
            assert y[row, head].isnan().all() and lse[row, head].isnan()
