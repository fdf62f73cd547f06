"""GPU test of keeping a path whose positions lie on an impossible page: reported, nothing moves and nothing is kept of
it, and the other sequences' paths are."""
import pytest
import torch

from test_paged_gpu import BF, F32, lla  # noqa: F401
from test_paged_pages_gpu import Pair, ints, pools

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [-1, 30, 2 ** 31 - 1])
@pytest.mark.parametrize("dtype,at,path,good", [
    (BF, 2, [0, 40, 41], False),   # a source
    (F32, 0, [20, 40], False),     # a destination
    (BF, 1, [10, 11, 40], True),   # neither
    (F32, 2, [0, 1, 2], True),     # nothing moves
])
def test_impossible_pages(lla, dtype, at, path, good, page):  # noqa: F811
    """Sequence 0 has 44 nodes from position 4 on (pages of 16: 0 is a destination, 2 holds nodes 28 to 43)."""
    pool = pools(30, dtype=dtype)
    rows = [[11, 12, 13], [14, 15, 16]]
    P = Pair(lla, rows, [48, 48], 3, pool)
    P.device.page_table[0, at] = page
    want = [x.clone() for x in pool]
    paths = [path + [-1] * (4 - len(path)), [3, 20, 43, -1]]
    for b, p in enumerate(paths):
        if b == 0 and not good:
            continue
        for x, y in zip(want, pool):
            for i, a in enumerate(p):
                if a >= 0 and a != i:
                    x[rows[b][(4 + i) // 16], :, (4 + i) % 16] = y[rows[b][(4 + a) // 16], :, (4 + a) % 16]
    keep = lla.lla_paged_compact(P.device, ints([0, 44, 88]), ints(paths))
    assert lla.lla_stream_status() == (0 if good else 1)
    assert keep.tolist() == [4 + len(path) * good, 7]
    assert all(torch.equal(x, y) for x, y in zip(pool, want))


def test_a_path_longer_than_the_nodes(lla):  # noqa: F811
    """It cannot rise throughout: refused without a look at the table behind the sequence's end."""
    pool = pools(30)
    P = Pair(lla, [[11, 12, 13]], [48], 3, pool)
    before = [x.clone() for x in pool]
    keep = lla.lla_paged_compact(P.device, ints([0, 6]), ints([[0, 1, 2, 3, 4, 5] + [1, 2, 3, 4, 5] * 400]))
    assert lla.lla_stream_status() == 1 and keep.tolist() == [42]
    assert all(torch.equal(x, y) for x, y in zip(pool, before))
