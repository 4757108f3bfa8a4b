"""PagePool against a model that keeps every request's tokens in a list: random
runs of adds, forks, writes, frees and compactions on a simulated cache, whose
pages are written and copied only as the pool says."""
import random

import numpy as np
import pytest

from linear_attention_blocked_b200.serving import PagePool, PoolExhausted


class Sim:
    def __init__(self, n_pages, page):
        self.pool, self.page = PagePool(n_pages, page), page
        self.cache = np.full((n_pages, page), -1, dtype=np.int64)
        self.tokens = {}
        self.clock = 0

    def copy(self, pairs):
        src, dst = pairs
        assert len(set(dst.tolist())) == len(dst) and not set(dst.tolist()) & set(src.tolist())
        self.cache[dst] = self.cache[src]

    def write(self, request, n):
        """One step of the request, its copies run first."""
        self.pool.reserve(request, n)
        self.copy(self.pool.take_copies())
        for _ in range(n):
            at = len(self.tokens[request])
            self.cache[self.pool.pages(request)[at // self.page], at % self.page] = self.clock
            self.tokens[request].append(self.clock)
            self.clock += 1
        self.pool.advance(request, n)

    def check(self):
        held = {}
        for r, want in self.tokens.items():
            assert self.pool.length(r) == len(want)
            pages = self.pool.pages(r)
            got = [int(self.cache[pages[i // self.page], i % self.page]) for i in range(len(want))]
            assert got == want
            for p in pages:
                held[p] = held.get(p, 0) + 1
        assert self.pool.free_pages == self.pool.n_pages - len(held)


@pytest.mark.parametrize("seed", range(8))
def test_random_runs_keep_every_request(seed):
    rng = random.Random(seed)
    sim = Sim(60, 16)
    for _ in range(400):
        do = rng.random()
        live = list(sim.tokens)
        try:
            if do < 0.15 or not live:
                sim.tokens[sim.pool.add()] = []
            elif do < 0.6:
                sim.write(rng.choice(live), rng.choice([0, 1, 1, 1, 5, 16, 40]))
            elif do < 0.75:
                parent = rng.choice(live)
                sim.tokens[sim.pool.fork(parent)] = list(sim.tokens[parent])
            elif do < 0.95:
                r = rng.choice(live)
                sim.pool.free(r)
                del sim.tokens[r]
                assert r not in sim.pool
            else:
                sim.copy(sim.pool.compact())
                used = {p for r in sim.tokens for p in sim.pool.pages(r)}
                assert used == set(range(len(used)))
        except PoolExhausted:
            pass
        sim.check()


def test_copies_of_a_batch_never_name_a_page_twice():
    """Reserves, frees and forks of one batch before its copies are taken."""
    rng = random.Random(5)
    for _ in range(200):
        pool = PagePool(30, 16)
        live = []
        for _ in range(3):
            r = pool.add()
            pool.reserve(r, 20)
            pool.advance(r, 20)
            live.append(r)
        live += [pool.fork(rng.choice(live)) for _ in range(5)]
        for _ in range(8):
            if rng.random() < 0.4 and len(live) > 1:
                pool.free(live.pop(rng.randrange(len(live))))
            else:
                try:
                    pool.reserve(rng.choice(live), 1)
                except PoolExhausted:
                    pass
        src, dst = pool.take_copies()
        assert len(set(dst.tolist())) == len(dst)
        assert not set(src.tolist()) & set(dst.tolist())
        held = {p for r in live for p in pool.pages(r)}
        assert pool.free_pages == 30 - len(held)


def test_exhausted_pool_changes_nothing():
    pool = PagePool(4, 16)
    a = pool.add()
    pool.reserve(a, 40)
    pool.advance(a, 40)
    b = pool.fork(a)
    before = (pool.pages(a), pool.pages(b), pool.free_pages)
    with pytest.raises(PoolExhausted):
        pool.reserve(b, 9 + 16)      # a copy of the ragged page and one more: two pages
    assert (pool.pages(a), pool.pages(b), pool.free_pages) == before
    pool.reserve(b, 8)
    src, dst = pool.take_copies()
    assert src.tolist() == [before[0][2]] and dst.tolist() == [pool.pages(b)[2]]


def test_tables_and_refusals():
    pool = PagePool(8, 32)
    a, b = pool.add(), pool.add()
    pool.reserve(a, 70)
    pool.advance(a, 65)
    assert pool.table([a, None, b]).shape == (3, 3)
    assert pool.table([a], max_pages=5)[0, :3].tolist() == pool.pages(a)
    assert pool.lengths([a, None, b]).tolist() == [65, -1, 0]
    assert pool.table([]).shape == (0, 1)
    with pytest.raises(ValueError):
        pool.table([a], max_pages=2)
    with pytest.raises(ValueError):
        pool.advance(a, 32)
    with pytest.raises(ValueError):
        pool.reserve(a, -1)
    with pytest.raises(ValueError):
        PagePool(8, 48)
    c = pool.fork(a)
    pool.reserve(c, 1)
    with pytest.raises(RuntimeError):
        pool.compact()
    pool.take_copies()
    pool.compact()


def test_fork_of_a_fork_before_its_copy_is_taken():
    """A page that a collected copy will fill is forked again: the second copy
    reads what the first one reads, and no page is both source and destination."""
    pool = PagePool(8, 16)
    a = pool.add()
    pool.reserve(a, 20)
    pool.advance(a, 20)
    b = pool.fork(a)
    pool.reserve(b, 1)
    c = pool.fork(b)
    pool.reserve(c, 1)
    d = pool.fork(c)
    pool.reserve(d, 30)
    src, dst = pool.take_copies()
    assert not set(src) & set(dst) and len(set(dst)) == len(dst)
    held = dict(zip(dst.tolist(), src.tolist()))
    for r in (b, c, d):
        assert held[pool.pages(r)[1]] == pool.pages(a)[1]
    assert len({pool.pages(r)[1] for r in (a, b, c, d)}) == 4
