"""A pool that runs out of pages while sequences of different lengths share a partly filled one: nobody's tokens are
written over."""
from __future__ import annotations

import random

import pytest
import torch

import quantized_gemv_gguf_amd as q
from test_gpu_kv import ints

pytestmark = pytest.mark.gpu


class Shared:
    """Sequence 1 holds the page of sequence 0, which was cut; a page's slots are token numbers."""

    def __init__(self, dev, lens, n_pages, size=16):
        n = len(lens)
        full = lambda shape, v: torch.full(shape, v, dtype=torch.int32, device=dev)  # noqa: E731
        self.dev = dev
        self.pool = q.KvPool(full((n, 4), -1), full((n,), 0), full((n_pages,), 0), full((1,), 0), size,
                             torch.empty(q.qgemv_kv_pool_bytes(n, 4, n_pages), dtype=torch.uint8, device=dev))
        self.cache = q.KvCache(*(torch.zeros(1, n_pages, 1, size, 32, dtype=torch.float16, device=dev) for _ in range(2)))
        self.resize([max(lens)] + [-1] * (n - 1))
        self.append(0, 0, max(lens), 100)
        q.qgemv_kv_fork(self.pool, ints([0] * n, dev))
        self.resize(lens)

    def resize(self, lens):
        q.qgemv_kv_resize(self.pool, self.cache, ints(lens, self.dev))
        return self.pool.lens.tolist()

    def append(self, s, first, end, value):
        """Token numbers value + position at the positions from `first` on of sequence s, of length `end`."""
        n = len(self.pool.lens)
        starts = [0] * (s + 1) + [end - first] * (n - s)
        x = (torch.arange(first, end, device=self.dev) + value).float().view(-1, 1, 1).expand(-1, 1, 32).contiguous()
        q.qgemv_kv_append(x, x, q.KvSeqs(ints(starts, self.dev), self.pool.lens, self.pool.tables), self.cache, 0)

    def tokens(self, s):
        n = int(self.pool.lens[s])
        at = torch.arange(n)
        return self.cache.k[0, self.pool.tables[s].cpu().long()[at // 16], 0, at % 16, 0].int().tolist()


def test_first_holder_does_not_write_over_a_longer_one(dev):
    """Both want to grow, and the second finds no page for its copy: the first, which is shorter, would keep the page
    and write its next token over the second's."""
    p = Shared(dev, [5, 8], 1)
    lens = p.resize([6, 9])
    assert lens == [5, 8]
    p.append(0, 4, lens[0], 200)  # (its last token again, its own)
    assert p.tokens(1) == [100, 101, 102, 103, 204, 105, 106, 107] and p.pool.refs.tolist() == [2]
    # with the second gone the first grows in place
    assert p.resize([-1, 0]) == [5, 0] and p.resize([6, -1]) == [6, 0]
    assert p.pool.tables.tolist() == [[0, -1, -1, -1], [-1] * 4] and p.pool.used.tolist() == [1]


@pytest.mark.parametrize("lens,want,pages,got", [
    ([8, 8], [9, 9], 1, [9, 8]),            # the same length: the first writes behind the second's end
    ([8, 5], [9, 6], 1, [9, 5]),            # so does a longer first
    ([5, 8], [6, 9], 2, [6, 9]),            # a page for the copy
    ([5, 8], [20, 9], 2, [5, 8]),           # the first takes the only one, stays, and gives it back
    ([5, 8, 5], [6, 9, 6], 2, [6, 9, 5]),   # the second finds a copy's page, the third, which is no longer, does not
    ([5, 5, 8], [6, 6, 9], 2, [5, 6, 8]),   # the third does not
    ([5, 8], [6, 40], 2, [5, 8]),           # a copy and more than there is
])
def test_full_pools(dev, lens, want, pages, got):
    p = Shared(dev, lens, pages)
    before = [p.tokens(s) for s in range(len(lens))]
    now = p.resize(want)
    assert now == got
    for s, (a, n) in enumerate(zip(lens, now)):
        if n > a:
            p.append(s, a, n, 200 + 50 * s)
    for s, (a, n) in enumerate(zip(lens, now)):
        assert p.tokens(s) == before[s] + [200 + 50 * s + i for i in range(a, n)], s
    refs = [0] * pages
    for row, n in zip(p.pool.tables.tolist(), now):
        held = -(-n // 16)
        assert row[held:] == [-1] * (4 - held)
        for page in row[:held]:
            refs[page] += 1
    assert p.pool.refs.tolist() == refs and p.pool.used.tolist() == [sum((r > 0) << i for i, r in enumerate(refs))]


@pytest.mark.parametrize("seed", range(16))
def test_steps_of_scarce_pages(dev, seed):
    """Random growth, cuts, forks and compaction of a pool that is often full: every sequence's tokens are its own
    history's, pages and counts as the tables have them."""
    r = random.Random(seed)
    n, size, wide = r.choice([2, 3, 5, 30]), r.choice([1, 4, 16]), r.choice([2, 5])
    pages = r.choice([2, n, n * wide // 2 + 1])
    full = lambda shape, v: torch.full(shape, v, dtype=torch.int32, device=dev)  # noqa: E731
    pool = q.KvPool(full((n, wide), -1), full((n,), 0), full((pages,), 0), full((-(-pages // 32),), 0), size,
                    torch.empty(q.qgemv_kv_pool_bytes(n, wide, pages), dtype=torch.uint8, device=dev))
    cache = q.KvCache(*(torch.zeros(1, pages, 1, size, 32, dtype=torch.float16, device=dev) for _ in range(2)))
    own, token = [[] for _ in range(n)], 0
    for step in range(20):
        kind = r.choice(["resize", "resize", "resize", "fork", "compact"])
        if kind == "fork":
            parents = [r.choice([s, s, -1, r.randrange(n), r.randrange(n)]) for s in range(n)]
            q.qgemv_kv_fork(pool, ints(parents, dev))
            own = [list(own[f]) if f >= 0 else [] for f in parents]
        elif kind == "compact":
            q.qgemv_kv_compact(pool, cache)
        else:
            want = [r.choice([len(h) + r.randint(1, size + 1), r.randint(0, len(h)), -1]) for h in own]
            q.qgemv_kv_resize(pool, cache, ints(want, dev))
            starts, new = [0], []
            for h, w, m in zip(own, want, pool.lens.tolist()):
                assert m == len(h) if w < 0 else m == w if w <= len(h) else m in (w, len(h))
                del h[m:]
                for _ in range(m - len(h)):
                    token = (token + 1) % 2048
                    new.append(token)
                    h.append(token)
                starts.append(len(new))
            if new:
                x = torch.tensor(new, dtype=torch.float32, device=dev).view(-1, 1, 1).expand(-1, 1, 32).contiguous()
                q.qgemv_kv_append(x, x, q.KvSeqs(ints(starts, dev), pool.lens, pool.tables), cache, 0)
        refs = [0] * pages
        for s, (h, row) in enumerate(zip(own, pool.tables.cpu())):
            at, held = torch.arange(len(h)), -(-len(h) // size)
            assert cache.k.cpu()[0, row.long()[at // size], 0, at % size, 3].tolist() == h, (step, kind, s)
            assert (row[held:] == -1).all()
            for page in row[:held].tolist():
                refs[page] += 1
        assert pool.lens.tolist() == [len(h) for h in own] and pool.refs.tolist() == refs
        word = [sum((x > 0) << i for i, x in enumerate(refs[w:w + 32])) for w in range(0, pages, 32)]
        assert [w & 0xffffffff for w in pool.used.tolist()] == word
