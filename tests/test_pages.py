"""The pages of a cache against a plain list implementation: tables, reference counts and copied pages, all exact."""
import random

import pytest
import torch

from gated_deltanet_linear_step_amd import ops

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


class Lists:
    """The operators on Python lists."""

    def __init__(self, table, refs, pool, ps):
        self.table, self.refs, self.pool, self.ps = table.tolist(), refs.tolist(), pool.clone(), ps
        self.width, self.pages = table.shape[1], len(self.refs)

    def is_page(self, p):
        return 0 <= p < self.pages

    def entries(self, n):
        e = -(-n // self.ps)
        return -1 if n < 0 or e > self.width else e

    def free(self, rows, keep=None):
        for i, r in enumerate(rows):
            if 0 <= r < len(self.table):
                for e in range(max(keep[i], 0) if keep else 0, self.width):
                    if self.is_page(self.table[r][e]):
                        self.refs[self.table[r][e]] -= 1
                    self.table[r][e] = -1

    def reserve(self, rows, lens):
        status, spent = [], False
        for i, (r, n) in enumerate(zip(rows, lens)):
            e = self.entries(n)
            if not 0 <= r < len(self.table) or e < 0 or r in rows[:i]:
                status.append(2)
                continue
            missing = [x for x in range(e) if not self.is_page(self.table[r][x])]
            open_ = [p for p in range(self.pages) if self.refs[p] <= 0]
            if missing and (spent or len(missing) > len(open_)):
                spent = True
                status.append(1)
                continue
            for x, p in zip(missing, open_):
                self.table[r][x], self.refs[p] = p, 1
            status.append(0)
        return status

    def fork(self, src, dst, lens):
        status, spent = [], False
        before = [list(r) for r in self.table]
        for i, (a, b, n) in enumerate(zip(src, dst, lens)):
            e = self.entries(n)
            bad = e < 0 or not 0 <= a < len(before) or not 0 <= b < len(before) or b in dst[:i] or a in dst
            bad = bad or any(not self.is_page(p) for p in before[a][:e]) or any(self.is_page(p) for p in before[b])
            if bad:
                status.append(2)
                continue
            full = n // self.ps
            if n % self.ps:
                open_ = [p for p in range(self.pages) if self.refs[p] <= 0]
                if spent or not open_:
                    spent = True
                    status.append(1)
                    continue
                self.table[b][full], self.refs[open_[0]] = open_[0], 1
                self.pool[:, open_[0]] = self.pool[:, before[a][full]]
            for x in range(full):
                self.table[b][x] = before[a][x]
                self.refs[before[a][x]] += 1
            status.append(0)
        return status

    def compact(self):
        used = sum(r > 0 for r in self.refs)
        to = list(range(self.pages))
        holes = iter([p for p in range(used) if self.refs[p] <= 0])
        for p in range(used, self.pages):
            if self.refs[p] > 0:
                to[p] = next(holes)
                self.pool[:, to[p]] = self.pool[:, p]
                self.refs[to[p]], self.refs[p] = self.refs[p], 0
        self.table = [[to[p] if self.is_page(p) else p for p in row] for row in self.table]
        return to, used


class Cache:
    """Both of them side by side."""

    def __init__(self, rows, width, pages, ps, planes=3, elems=40, pad=(0, 0), seed=1):
        gen = torch.Generator(DEV).manual_seed(seed)
        big = torch.randint(-2 ** 15, 2 ** 15, (planes, pages + pad[0], elems + pad[1]), dtype=torch.int16, device=DEV, generator=gen)
        self.big, self.pool = big, big[:, :pages, :elems]
        self.table = torch.full((rows, width + 2), -1, dtype=torch.int32, device=DEV)[:, :width]
        self.refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
        self.ps, self.want = ps, Lists(self.table, self.refs, self.pool, ps)
        self.beside = big.clone()

    @staticmethod
    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def check(self):
        torch.cuda.synchronize()
        assert self.table.tolist() == self.want.table
        assert self.refs.tolist() == self.want.refs
        assert torch.equal(self.pool, self.want.pool)
        assert torch.equal(self.big[:, self.pool.shape[1]:], self.beside[:, self.pool.shape[1]:])
        assert torch.equal(self.big[:, :, self.pool.shape[2]:], self.beside[:, :, self.pool.shape[2]:])

    def free(self, rows, keep=None):
        ops.pages_free(self.table, self.refs, self.i32(rows), keep=None if keep is None else self.i32(keep))
        self.want.free(rows, keep)
        self.check()

    def reserve(self, rows, lens):
        got = ops.pages_reserve(self.table, self.refs, self.i32(rows), self.i32(lens), page_size=self.ps)
        status = self.want.reserve(rows, lens)
        self.check()
        assert got.tolist() == status
        return status

    def fork(self, src, dst, lens):
        got = ops.pages_fork(self.pool, self.table, self.refs, self.i32(src), self.i32(dst), self.i32(lens), page_size=self.ps)
        status = self.want.fork(src, dst, lens)
        self.check()
        assert got.tolist() == status
        return status

    def compact(self):
        got = ops.pages_compact(self.pool, self.table, self.refs)
        to, used = self.want.compact()
        self.check()
        assert got[0].tolist() == to and got[1].tolist() == [used]


def test_a_cache_through_its_life():
    c = Cache(rows=8, width=6, pages=20, ps=4, pad=(3, 8))
    assert c.reserve([0, 3, 5], [9, 0, 24]) == [0, 0, 0]
    assert c.reserve([0, 3], [13, 1]) == [0, 0]          # a row grows
    assert c.fork([0, 0, 5], [1, 2, 4], [13, 12, 24]) == [0, 0, 0]
    c.free([0])                                          # shared pages stay
    assert c.fork([1, 1], [0, 7], [2, 0]) == [0, 0]
    c.free([5, 1], [2, 0])
    c.compact()
    c.free([0, 1, 2, 3, 4, 5, 6, 7])
    assert c.refs.sum() == 0
    c.compact()


def test_requests_that_are_refused():
    c = Cache(rows=5, width=4, pages=8, ps=4)
    assert c.reserve([0, 9, -1, 0, 1, 2, 3], [16, 4, 4, 4, -1, 17, 2 ** 31 - 1]) == [0, 2, 2, 2, 2, 2, 2]
    # no source pages, a source that is a destination, a full destination, rows out of range, a destination twice; row 0,
    # which the third names as its destination, serves none as a source
    assert c.fork([1, 2, 1, 0, 0, 0, 0, 9], [2, 3, 0, 1, 1, -1, 5, 4], [4, 4, 0, 5, 5, 4, 4, 4]) == [2, 2, 2, 2, 2, 2, 2, 2]
    assert c.fork([0, 0, 0, 0, 9, 2], [1, 1, -1, 5, 4, 3], [5, 5, 4, 4, 4, 4]) == [0, 2, 2, 2, 2, 2]
    c.free([9, -1, 2 ** 31 - 1, 1, 1], [0, 0, 0, 1, 0])
    c.free([0], [2 ** 31 - 1])
    c.free([0], [-7])


def test_pages_that_run_out():
    c = Cache(rows=6, width=8, pages=10, ps=2)
    assert c.reserve([0, 1, 2, 3], [8, 9, 4, 0]) == [0, 0, 1, 0]
    assert c.reserve([2], [2]) == [0]
    assert c.fork([0, 0, 1], [3, 4, 5], [4, 3, 9]) == [0, 1, 1]
    c.free([1])
    assert c.fork([0, 0], [4, 5], [3, 3]) == [0, 0]


def test_entries_that_are_no_pages():
    c = Cache(rows=3, width=5, pages=6, ps=4)
    c.reserve([0], [12])
    for x, bad in ((1, -5), (4, 10 ** 9)):
        c.table[0, x] = bad
        c.want.table[0][x] = bad
    assert c.fork([0], [1], [9]) == [2]
    assert c.fork([0], [1], [3]) == [0]
    c.compact()
    assert c.reserve([0], [12]) == [0]
    c.free([0])


@pytest.mark.parametrize("seed", range(6))
def test_random_lives(seed):
    rng = random.Random(seed)
    ps, width = rng.choice((1, 3, 16)), rng.choice((3, 70, 150))
    rows, pages = rng.choice((5, 40)), rng.choice((30, 900, 9000))
    c = Cache(rows, width, pages, ps, planes=2, elems=8, seed=seed)
    for _ in range(25):
        n = rng.randrange(1, rows + 1)
        some = rng.sample(range(rows), n)
        lens = [rng.randrange(0, ps * width + 1) for _ in range(n)]
        kind = rng.randrange(4)
        if kind == 0:
            c.free(some, rng.choice((None, [rng.randrange(0, width) for _ in some])))
        elif kind == 1:
            c.reserve(some, lens)
        elif kind == 2:
            have = [next((e for e in range(width) if not c.want.is_page(c.want.table[r][e])), width) * ps for r in range(rows)]
            empty = [r for r in range(rows) if have[r] == 0]
            full = [r for r in range(rows) if have[r] > 0]
            if empty and full:
                src = [rng.choice(full) for _ in empty]
                c.fork(src, empty, [rng.randrange(0, have[r] + 1) for r in src])
        else:
            c.compact()


@pytest.mark.parametrize("n", [1, 64, 65, 1024])
def test_many_requests(n):
    c = Cache(rows=2 * n + 1, width=3, pages=3 * n + 70, ps=16, planes=1, elems=8)
    c.reserve([2 * n], [40])
    c.fork([2 * n] * n, list(range(n)), [17 + i % 16 for i in range(n)])
    c.reserve(list(range(n, 2 * n)), [20] * n)
    c.free(list(range(0, 2 * n, 2)))
    c.compact()


def test_requests_for_thousands_of_pages():
    c = Cache(rows=4, width=6000, pages=20000, ps=1, planes=1, elems=8)
    c.reserve([0, 1, 2], [5000, 4097, 1])
    c.free([0], [10])
    c.reserve([0, 3], [6000, 6000])
    c.fork([3], [2], [6000])   # row 2 is not empty
    c.free([2, 1])
    c.fork([3], [2], [6000])
    c.compact()


@pytest.mark.parametrize("page_elems", [8, 1000, 8192, 8200, 100000])
def test_pages_of_any_size(page_elems):
    c = Cache(rows=4, width=5, pages=12, ps=16, planes=4, elems=page_elems, pad=(1, 16))
    c.reserve([3], [70])
    c.reserve([0], [70])
    c.free([3])
    c.fork([0, 0], [1, 2], [69, 33])
    c.free([0])
    c.compact()


def test_captured_calls_and_their_own_stream():
    c = Cache(rows=6, width=5, pages=16, ps=4, planes=2, elems=16)
    c.reserve([0, 1], [18, 7])
    table0, refs0, pool0 = c.table.clone(), c.refs.clone(), c.pool.clone()
    i32 = c.i32
    src, dst, lens, rows = i32([0, 0, 1]), i32([2, 3, 4]), i32([18, 9, 7]), i32([0, 3])

    def life(stream=None):
        status = ops.pages_fork(c.pool, c.table, c.refs, src, dst, lens, page_size=4, stream=stream)
        ops.pages_free(c.table, c.refs, rows, stream=stream)
        more = ops.pages_reserve(c.table, c.refs, rows, lens[:2], page_size=4, stream=stream)
        ops.pages_free(c.table, c.refs, rows[:1], stream=stream)
        return status, more, *ops.pages_compact(c.pool, c.table, c.refs, stream=stream)

    got = life()
    want = [t.clone() for t in (c.table, c.refs, c.pool, *got)]

    def reset():
        c.table.copy_(table0), c.refs.copy_(refs0), c.pool.copy_(pool0)
        torch.cuda.synchronize()

    reset()
    stream = torch.cuda.Stream()
    got = life(stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((c.table, c.refs, c.pool, *got), want))
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = life()
    for _ in range(3):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((c.table, c.refs, c.pool, *got), want))


def test_planes_past_32_bits():
    """Pages and planes whose byte offsets pass 2^32."""
    pages, elems, far = 6, 16, 1 << 29  # int16 elements from page to page
    buf = torch.zeros(2 * pages * far, dtype=torch.int16, device=DEV)
    pool = buf.as_strided((2, pages, elems), (pages * far, far, 1))
    pool.copy_(torch.randint(1, 1000, (2, pages, elems), dtype=torch.int16, device=DEV))
    start = pool.clone()
    table = torch.tensor([[5, 4, -1], [-1, -1, -1]], dtype=torch.int32, device=DEV)
    refs = torch.tensor([0, 0, 0, 0, 1, 1], dtype=torch.int32, device=DEV)
    i32 = Cache.i32
    assert ops.pages_fork(pool, table, refs, i32([0]), i32([1]), i32([5]), page_size=4).tolist() == [0]
    assert table.tolist() == [[5, 4, -1], [5, 0, -1]] and torch.equal(pool[:, 0], start[:, 4])
    ops.pages_compact(pool, table, refs)
    assert table.tolist() == [[2, 1, -1], [2, 0, -1]] and refs.tolist() == [1, 1, 2, 0, 0, 0]
    assert torch.equal(pool[:, 1], start[:, 4]) and torch.equal(pool[:, 2], start[:, 5])
