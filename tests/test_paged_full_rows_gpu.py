"""GPU tests of sequences that would outgrow their row of the table: grow changes nothing and says so in `left`, where
its caller looks before anything is appended. Whole numbers and moved values: exact."""
import pytest
import torch

from paged_pages_reference import Book
from test_paged_gpu import BF, lla  # noqa: F401
from test_paged_pages_gpu import Pair, ints, pools, starts_of

pytestmark = pytest.mark.gpu


def state(P, refs):
    return P.device.lens.tolist(), P.device.page_table.tolist(), refs.tolist()


@pytest.mark.parametrize("news,left", [
    ([1, 1], -1),           # the first is full to the last slot
    ([0, 30], -1),          # 18 + 30 = 48 are three pages and fit; one more would not
    ([0, 31], -1),
    ([16, 0], -1), ([17, 0], -2), ([48, 0], -3),
    ([20, 33], -3),         # two entries of the first, one of the second
    ([0, 0], 5)])
def test_a_full_row_lets_nothing_change(lla, news, left):  # noqa: F811
    pool = pools(10)
    P = Pair(lla, [[3, 4, 5], [6, 7]], [48, 18], 3, pool)
    refs = ints([0, 0, 0, 1, 1, 1, 1, 1, 0, 0])
    if news == [0, 30]:
        left = 4
    before = state(P, refs)
    copies, got = lla.lla_paged_grow(P.device, starts_of(news), refs)
    assert got.tolist() == [left] and copies.tolist() == [[-1, -1]] * 2
    if left < 0 or not any(news):
        assert state(P, refs) == before
    else:
        assert P.device.lens.tolist() == [48, 48] and P.device.page_table.tolist()[1] == [6, 7, 0]
    assert lla.lla_stream_status() == 0


def test_pages_and_entries_that_lack_are_added_up(lla):  # noqa: F811
    pool = pools(8)
    P = Pair(lla, [[0, 1, 2], [3], [4]], [40, 16, 16], 3, pool)
    refs = ints([1, 1, 1, 1, 1, 1, 1, 0])
    before = state(P, refs)
    # one page is free; the last two take two each: three are missing; the first lacks one entry
    copies, left = lla.lla_paged_grow(P.device, starts_of([24, 32, 32]), refs)
    assert left.tolist() == [-4] and (copies == -1).all() and state(P, refs) == before
    assert lla.lla_stream_status() == 0


@pytest.mark.parametrize("B", [2, 40, 2000])
def test_grow_then_append_leaves_shared_positions(lla, B):  # noqa: F811
    """Every sequence holds the same pages, one row is full: a server that appends where left allows it writes over
    nothing that is there."""
    page, width = 16, 4
    pool = pools(3 * B + 8, mass=False)
    book = Book(3 * B + 8, page)
    full, most = list(range(width)), width * page
    lens = [most - 3] * B
    lens[B // 2] = most
    for _ in range(B):
        for x in full:
            book.refs[x] += 1
    P = Pair(lla, [list(full) for _ in range(B)], list(lens), width, pool)
    refs = ints(book.refs)
    before, held = state(P, refs), [x.clone() for x in pool[:2]]
    starts = starts_of([2] * B)
    copies, left = lla.lla_paged_grow(P.device, starts, refs)
    lla.lla_paged_copy(P.device, P.device, copies)
    if int(left) >= 0:
        k, v = (torch.zeros(2 * B, *x.shape[1:2], x.shape[3], dtype=BF, device="cuda") for x in pool[:2])
        lla.lla_paged_append(k, v, P.device, starts)
    assert all(torch.equal(x[:width], y[:width]) for x, y in zip(pool, held))
    assert left.tolist() == [-1] and state(P, refs) == before
    assert lla.lla_stream_status() == 0


def test_who_is_left_out_is_marked(lla):  # noqa: F811
    """Impossible lengths and starts: reported, marked, and the others grow."""
    pool = pools(20)
    P = Pair(lla, [[3, 4, 5], [6], [7, 8], [9]], [49, 9, 32, 3], 3, pool)
    refs = ints([0, 0, 0, 1, 1, 1, 1, 1, 1, 2] + [0] * 10)
    copies, left = lla.lla_paged_grow(P.device, ints([0, 1, 8, 57, 58]), refs)
    assert lla.lla_stream_status() == 1
    assert copies.tolist() == [[-2, -2], [-1, -1], [-2, -2], [9, 0]] and left.tolist() == [12]
    assert P.device.lens.tolist() == [49, 16, 32, 4]
    copies, left = lla.lla_paged_grow(P.device, ints([0, 0, 5, 4, 4]), refs)
    assert lla.lla_stream_status() == 1
    assert copies.tolist() == [[-2, -2], [-1, -1], [-2, -2], [-1, -1]]


def test_no_table_is_too_wide(lla):  # noqa: F811
    """A row of 2^30 - 16 positions: the sums pass 2^31."""
    max_pages = (1 << 26) - 1
    pool = pools(4, Hkv=1, page=16, d=16, dv=16, mass=False)
    wide = torch.zeros(1, max_pages, dtype=torch.int32, device="cuda")
    most = max_pages * 16
    cache = lla.PagedCache(pool[0], pool[1], wide, ints([most - 1]))
    refs = ints([1, 0, 0, 0])
    copies, left = lla.lla_paged_grow(cache, ints([0, most]), refs)
    assert left.tolist() == [-max_pages] and copies.tolist() == [[-1, -1]]
    assert cache.lens.tolist() == [most - 1] and lla.lla_stream_status() == 0


def grown(book, rows, lens, news, width):
    """The rules: (copies, left), rows and lens changed where there is room for all."""
    over = sum(max(0, book.pages(n + t) - width) for n, t in zip(lens, news))
    within = [min(t, width * book.page - n) for n, t in zip(lens, news)]
    trial = Book(0, book.page)
    trial.refs = list(book.refs)
    trial_rows, trial_lens = [list(r) for r in rows], list(lens)
    copies, left = trial.grow(trial_rows, trial_lens, within)
    if over:
        return [[-1, -1]] * len(lens), min(left, 0) - over
    if left >= 0:
        book.refs, rows[:], lens[:] = trial.refs, trial_rows, trial_lens
    return copies, left


@pytest.mark.parametrize("page,num_pages,B,width,seed", [(16, 40, 3, 4, 0), (32, 300, 33, 3, 1), (16, 2000, 500, 5, 2), (64, 90, 8, 9, 3),
                                                         (16, 9000, 4096, 2, 4)])
def test_any_order_with_narrow_tables(lla, page, num_pages, B, width, seed):  # noqa: F811
    """Rows that fill up, pools that run out, forks and shorter sequences, step after step."""
    import random
    rng = random.Random(seed)
    pool = pools(num_pages, Hkv=1, page=page, d=16, dv=16, mass=False)
    book, refs = Book(num_pages, page), torch.zeros(num_pages, dtype=torch.int32, device="cuda")
    cur, old = (Pair(lla, [[] for _ in range(B)], [0] * B, width, pool) for _ in range(2))
    seen = set()
    for step in range(40):
        kind = rng.choice(["grow", "grow", "grow", "fork", "keep"])
        if kind == "grow" or step % 10 == 9 and any(cur.lens):  # then one position more than a row has
            most = rng.choice([1, 2, page, width * page])
            news = [rng.choice([0, 1, rng.randint(0, most)]) if rng.random() < 8 / B else 0 for _ in range(B)]
            if rng.random() < 0.6:  # a step that fits its rows
                news = [min(t, width * page - n) for t, n in zip(news, cur.lens)]
            if step % 10 == 9 and any(cur.lens):
                b = next(b for b, n in enumerate(cur.lens) if n)
                news[b] = width * page - cur.lens[b] + 1
            full = any(n + t > width * page for n, t in zip(cur.lens, news))
            copies, left = lla.lla_paged_grow(cur.device, starts_of(news), refs)
            want, want_left = grown(book, cur.rows, cur.lens, news, width)
            assert copies.tolist() == want and left.tolist() == [want_left]
            seen.add((want_left < 0, full))
        elif kind == "fork":
            parents = [rng.randrange(-1, B) if rng.random() < 0.5 else rng.randrange(max(1, B // 4)) for _ in range(B)]
            lla.lla_paged_fork(cur.device, old.device, ints(parents), refs)
            old.rows, old.lens = book.fork(cur.rows, cur.lens, parents)
            lla.lla_paged_free(cur.device, refs)
            book.free(cur.rows, cur.lens)
            cur, old = old, cur
        else:
            keep = [rng.randint(-2, n + 3) if rng.random() < 0.2 else n for n in cur.lens]
            lla.lla_paged_free(cur.device, refs, ints(keep))
            book.free(cur.rows, cur.lens, keep)
        cur.check(book, refs)
        old.check(book, refs)
    assert lla.lla_stream_status() == 0
    assert {(False, False), (True, True)} <= seen
