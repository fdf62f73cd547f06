"""GPU tests of fork, free, grow, copy and compact against the rules on lists (paged_pages_reference.py). All of it is
exact: whole numbers and moved values."""
import random

import pytest
import torch

from paged_pages_reference import Book, table
from test_paged_gpu import BF, F32, lla  # noqa: F401

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts_of(news):
    return ints([sum(news[:b]) for b in range(len(news) + 1)])


class Pair:
    """Sequences on the device and on lists."""

    def __init__(self, lla, rows, lens, width, pools):  # noqa: F811
        self.rows, self.lens, self.width = rows, lens, width
        self.device = lla.PagedCache(pools[0], pools[1], table(rows, width).cuda(), ints(lens), pools[2])

    def check(self, book, refs):
        assert self.device.lens.tolist() == self.lens
        got = self.device.page_table.tolist()
        for b, row in enumerate(self.rows):
            assert got[b][:len(row)] == row, b
        assert refs.tolist() == book.refs


def pools(num_pages, Hkv=2, page=16, d=16, dv=32, dtype=BF, mass=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return [rnd(num_pages, Hkv, page, d).to(dtype), rnd(num_pages, Hkv, page, dv).to(dtype),
            rnd(num_pages, Hkv, page) if mass else None]


@pytest.mark.parametrize("page,num_pages,B,seed", [(16, 60, 3, 0), (16, 501, 9, 1), (64, 2048, 40, 2), (32, 1503, 130, 3),
                                                   (16, 40, 1, 4)])
def test_any_order_of_calls(lla, page, num_pages, B, seed):  # noqa: F811
    """Growing, forking onto the other table, shortening and running out, step after step."""
    rng = random.Random(seed)
    pool = pools(num_pages, page=page)
    book, refs = Book(num_pages, page), torch.zeros(num_pages, dtype=torch.int32, device="cuda")
    width = max(4, 3 * num_pages // B)
    cur = Pair(lla, [[] for _ in range(B)], [0] * B, width, pool)
    old = Pair(lla, [[] for _ in range(B)], [0] * B, width, pool)
    ran_out = False
    for step in range(60):
        kind = rng.choice(["grow", "grow", "grow", "grow", "fork", "fork", "keep"])
        if kind == "grow" or step == 30:  # then more than there is
            most = rng.choice([1, page, 6 * page, width * page])
            news = [rng.choice([0, 1, rng.randint(0, most)]) for _ in range(B)]
            news = [width * page - n if step == 30 else min(t, width * page - n) for t, n in zip(news, cur.lens)]
            copies, left = lla.lla_paged_grow(cur.device, starts_of(news), refs)
            want, want_left = book.grow(cur.rows, cur.lens, news)
            assert copies.tolist() == want and left.tolist() == [want_left]
            ran_out |= want_left < 0
        elif kind == "fork":
            parents = [rng.randrange(-1, B) if rng.random() < 0.5 else rng.randrange(max(1, B // 4)) for _ in range(B)]
            lla.lla_paged_fork(cur.device, old.device, ints(parents), refs)
            old.rows, old.lens = book.fork(cur.rows, cur.lens, parents)
            lla.lla_paged_free(cur.device, refs)
            book.free(cur.rows, cur.lens)
            cur, old = old, cur
        else:
            keep = None if rng.random() < 0.1 else [rng.randint(-2, n + 3) if rng.random() < 0.3 else n for n in cur.lens]
            lla.lla_paged_free(cur.device, refs, None if keep is None else ints(keep))
            book.free(cur.rows, cur.lens, keep)
        cur.check(book, refs)
        old.check(book, refs)
    assert lla.lla_stream_status() == 0
    assert ran_out


@pytest.mark.parametrize("B,num_pages", [(1, 1), (1, 127), (2, 128), (300, 4001), (1030, 200003), (4096, 9001)])
def test_grow_finds_the_lowest_pages(lla, B, num_pages):  # noqa: F811
    """Counts of any pattern, the pool just large enough, then too small; sequences that share a last page and grow, one or more of
    them, with or without others that hold it."""
    rng = random.Random(B + num_pages)
    page, book = 16, Book(num_pages, 16)
    pool = pools(num_pages, Hkv=1, dv=16, mass=False)
    shared = rng.sample(range(num_pages), min(num_pages // 3, max(1, B // 3)))
    rows, lens = [], []
    for b in range(B):
        n = rng.randint(1, 30) if num_pages > 3 * B else rng.choice([0, 5])
        row = [rng.choice(shared) for _ in range(-(-n // page))] if shared else []
        rows.append(row)
        lens.append(n if shared else 0)
        for x in row:
            book.refs[x] += 1
    for x in range(num_pages):
        if book.refs[x] == 0 and rng.random() < 0.6:
            book.refs[x] = rng.randint(1, 3)
    spare = book.refs.count(0)
    news = [rng.choice([0, 1, 12, 40]) if num_pages > 3 * B else rng.choice([0, 0, 1]) for _ in range(B)]
    for extra in (0, 1):
        refs = ints(book.refs)
        P = Pair(lla, [list(r) for r in rows], list(lens), 6, pool)
        trial = Book(num_pages, page)
        trial.refs = list(book.refs)
        used = len(spare_needed(trial, P, news))
        if extra:  # occupy all but one too few
            at = [x for x, c in enumerate(trial.refs) if c == 0]
            for x in at[max(0, used - 1):]:
                trial.refs[x] = 1
            refs = ints(trial.refs)
        copies, left = lla.lla_paged_grow(P.device, starts_of(news), refs)
        want, want_left = trial.grow(P.rows, P.lens, news)
        assert copies.tolist() == want and left.tolist() == [want_left]
        assert (want_left >= 0) == (used <= spare if not extra else used == 0)
        P.check(trial, refs)
    assert lla.lla_stream_status() == 0


def spare_needed(book, P, news):
    trial = Book(len(book.refs), book.page)
    trial.refs = list(book.refs) + [0] * 100000
    rows, lens = [list(r) for r in P.rows], list(P.lens)
    before = trial.refs.count(0)
    _, left = trial.grow(rows, lens, news)
    return range(before - left)


@pytest.mark.parametrize("dtype,Hkv,page,d,dv,mass", [(BF, 8, 64, 128, 128, True), (F32, 1, 16, 16, 64, False),
                                                      (BF, 3, 256, 64, 32, True), (F32, 2, 32, 128, 16, True), (BF, 1, 16, 16, 16, False)])
def test_copy(lla, dtype, Hkv, page, d, dv, mass):  # noqa: F811
    n, m = 30, 45
    a, b = pools(n, Hkv, page, d, dv, dtype, mass), pools(m, Hkv, page, d, dv, dtype, True, seed=1)
    one = lambda p: lla.PagedCache(*p[:2], ints([[0]]), ints([0]), p[2])  # noqa: E731
    src, dst = one(a), one(b)
    pairs = [[0, 44], [29, 0], [5, 7], [5, 8], [-1, 3], [4, -1], [-1, -1]]
    want = [x.clone() for x in b]
    for i, j in pairs:
        if i >= 0 and j >= 0:
            for x, y in zip(want, a):
                if y is not None:
                    x[j] = y[i]
    lla.lla_paged_copy(src, dst, ints(pairs))
    assert lla.lla_stream_status() == 0
    assert all(torch.equal(x, y) for x, y in zip(b, want))
    inside = [x.clone() for x in b]
    lla.lla_paged_copy(dst, dst, ints([[1, 2], [3, 4], [44, 43]]))
    for x, y in zip(b, inside):
        y[[2, 4, 43]] = y[[1, 3, 44]]
        assert torch.equal(x, y)
    lla.lla_paged_copy(src, dst, ints([[n, 1], [0, m], [6, 9]]))
    assert lla.lla_stream_status() == 1
    for x, y, z in zip(b, inside, a):
        if z is not None:
            y[9] = z[6]
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype,Hkv,page,d,dv,mass", [(BF, 8, 64, 128, 128, True), (F32, 1, 16, 16, 64, False), (F32, 2, 16, 128, 128, True),
                                                      (BF, 3, 256, 64, 32, True), (BF, 1, 16, 16, 16, False), (BF, 2, 16, 16, 128, True)])
@pytest.mark.parametrize("news,max_path", [([1], 1), ([12, 0, 5], 6), ([64, 7, 1, 30], 13), ([300, 120], 300)])
def test_compact(lla, dtype, Hkv, page, d, dv, mass, news, max_path):  # noqa: F811
    rng = random.Random(page + max_path)
    B = len(news)
    lens = [rng.randint(0, 90) + t for t in news]
    rows = [[] for _ in news]
    num_pages = sum(-(-n // page) for n in lens) + 3
    order = rng.sample(range(num_pages), num_pages)
    for b, n in enumerate(lens):
        rows[b] = [order.pop() for _ in range(-(-n // page))]
    pool = pools(num_pages, Hkv, page, d, dv, dtype, mass)
    P = Pair(lla, rows, list(lens), 40, pool)
    paths = [sorted(rng.sample(range(t), rng.randint(0, min(t, max_path)))) for t in news]
    paths[0] = sorted(rng.sample(range(news[0]), min(news[0], max_path)))
    want = [x.clone() for x in pool if x is not None]
    for b, path in enumerate(paths):
        first = lens[b] - news[b]
        for x, y in zip(want, pool):
            for i, a in enumerate(path):
                i_, a_ = first + i, first + a
                x[rows[b][i_ // page], :, i_ % page] = y[rows[b][a_ // page], :, a_ % page]
    keep = lla.lla_paged_compact(P.device, starts_of(news), ints([p + [-1] * (max_path - len(p)) for p in paths]))
    assert lla.lla_stream_status() == 0
    assert keep.tolist() == [n - t + len(p) for n, t, p in zip(lens, news, paths)]
    assert all(torch.equal(x, y) for x, y in zip([x for x in pool if x is not None], want))
    assert P.device.lens.tolist() == lens


def test_what_is_impossible_is_reported_and_left(lla):  # noqa: F811
    pool = pools(20)
    make = lambda: (Pair(lla, [[3, 4], [5], [6, 7]], [20, 9, 32], 3, pool), ints([0, 0, 0, 1, 1, 1, 1, 1] + [0] * 12))  # noqa: E731
    status = lla.lla_stream_status
    # fork: parents out of range, a length the table cannot hold, a target too narrow, a bad page number
    P, refs = make()
    to = Pair(lla, [[], [], [], []], [9, 9, 9, 9], 3, pool)
    P.device.lens[1] = 1000
    lla.lla_paged_fork(P.device, to.device, ints([3, 0, -2, 1]), refs)
    assert status() == 1 and to.device.lens.tolist() == [0, 20, 0, 0]
    assert refs.tolist()[3:8] == [2, 2, 1, 1, 1]
    narrow = Pair(lla, [[], []], [0, 0], 1, pool)
    P, refs = make()
    lla.lla_paged_fork(P.device, narrow.device, ints([0, 1]), refs)
    assert status() == 1 and narrow.device.lens.tolist() == [0, 9] and refs.tolist()[3:8] == [1, 1, 2, 1, 1]
    # free: an impossible length, a page that nobody holds
    P, refs = make()
    P.device.lens[0] = -1
    refs[5] = 0
    lla.lla_paged_free(P.device, refs)
    assert status() == 1 and P.device.lens.tolist() == [-1, 0, 0] and refs.tolist()[3:8] == [1, 1, 0, 0, 0]
    # grow: starts that descend, a length beyond the table, more than the table holds; the others grow
    P, refs = make()
    P.device.lens[0] = 49
    copies, left = lla.lla_paged_grow(P.device, ints([0, 1, 8, 100]), refs)
    assert status() == 1 and P.device.lens.tolist() == [49, 16, 32] and left.tolist() == [15]
    P, refs = make()
    lla.lla_paged_grow(P.device, ints([0, 12, 10, 11]), refs)
    assert status() == 1 and P.device.lens.tolist() == [32, 9, 33] and P.device.page_table[2].tolist() == [6, 7, 0]
    # compact: paths that do not rise or leave the nodes; impossible starts
    for bad in ([1, 1, -1], [2, 1, -1], [0, 4, -1]):
        P, refs = make()
        before = [x.clone() for x in pool]
        keep = lla.lla_paged_compact(P.device, ints([0, 4, 8, 12]), ints([bad, [-1, 0, 0], [0, 1, 2]]))
        assert status() == 1 and keep.tolist() == [16, 5, 31]
        assert all(torch.equal(x, y) for x, y in zip(pool, before))
    P, refs = make()
    keep = lla.lla_paged_compact(P.device, ints([0, 4, 2, 6]), ints([[-1], [-1], [-1]]))
    assert status() == 1 and keep.tolist() == [16, 9, 28]
    P.device.lens[0] = 500
    keep = lla.lla_paged_compact(P.device, ints([-3, -3, 0, 0]), ints([[0], [0], [-1]]))
    assert status() == 1 and keep.tolist()[2] == 32


def test_captured_and_on_another_stream(lla):  # noqa: F811
    """A beam step as one graph, replayed twice: each replay forks what the last one left."""
    page, num_pages, B = 16, 200, 6
    pool = pools(num_pages, page=page)
    book, refs = Book(num_pages, page), torch.zeros(num_pages, dtype=torch.int32, device="cuda")
    a, b = (Pair(lla, [[] for _ in range(B)], [0] * B, 10, pool) for _ in range(2))
    side = torch.cuda.Stream()
    first = starts_of([37] * B)
    copies, left = lla.lla_paged_grow(a.device, first, refs)
    book.grow(a.rows, a.lens, [37] * B)
    torch.cuda.synchronize()
    parents, news = ints([0, 0, 0, 3, 5, 5]), starts_of([1] * B)
    graph = torch.cuda.CUDAGraph()

    def step():
        for x, y in ((a, b), (b, a)):
            lla.lla_paged_fork(x.device, y.device, parents, refs)
            lla.lla_paged_free(x.device, refs)
            lla.lla_paged_grow(y.device, news, refs, copies, left)
            lla.lla_paged_copy(y.device, y.device, copies)
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(2):
        graph.replay()
        for x, y in ((a, b), (b, a)):
            y.rows, y.lens = book.fork(x.rows, x.lens, [0, 0, 0, 3, 5, 5])
            book.free(x.rows, x.lens)
            want, want_left = book.grow(y.rows, y.lens, [1] * B)
        torch.cuda.synchronize()
        a.check(book, refs)
        b.check(book, refs)
        assert copies.tolist() == want and left.tolist() == [want_left]
    got, left = lla.lla_paged_grow(a.device, news, refs, stream=side)
    side.synchronize()
    want, want_left = book.grow(a.rows, a.lens, [1] * B)
    assert got.tolist() == want and left.tolist() == [want_left]
    a.check(book, refs)
    assert lla.lla_stream_status() == 0


def test_no_sequences(lla):  # noqa: F811
    pool = pools(10)
    refs = ints([0, 1] * 5)
    empty = lla.PagedCache(pool[0], pool[1], ints([[]] * 0).reshape(0, 4), ints([]), pool[2])
    some = Pair(lla, [[1]], [3], 2, pool)
    copies, left = lla.lla_paged_grow(empty, ints([0]), refs)
    assert copies.shape == (0, 2) and left.tolist() == [5]
    lla.lla_paged_free(empty, refs)
    lla.lla_paged_fork(some.device, empty, ints([]), refs)
    lla.lla_paged_fork(empty, some.device, ints([-1]), refs)
    lla.lla_paged_copy(empty, empty, ints([]).reshape(0, 2))
    assert some.device.lens.tolist() == [0] and refs.tolist() == [0, 1] * 5 and lla.lla_stream_status() == 0


def test_grow_beyond_all_numbers(lla):  # noqa: F811
    """Starts that go up and down (reported) ask for 2^31 pages and more in all: nothing changes."""
    B, max_pages, page = 80, (1 << 26) - 1, 16
    pool = pools(4, Hkv=1, page=page, d=16, dv=16, mass=False)
    wide = torch.empty(B, max_pages, dtype=torch.int32, device="cuda")
    cache = lla.PagedCache(pool[0], pool[1], wide, torch.zeros(B, dtype=torch.int32, device="cuda"))
    refs = ints([0, 1, 0, 0])
    most = max_pages * page
    copies, left = lla.lla_paged_grow(cache, ints([0 if b % 2 == 0 else most for b in range(B + 1)]), refs)
    assert lla.lla_stream_status() == 1
    assert left.tolist() == [max(3 - 40 * max_pages, -2 ** 31 + 1)]
    assert (copies == -1).all() and (cache.lens == 0).all() and refs.tolist() == [0, 1, 0, 0]
