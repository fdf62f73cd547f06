"""GPU test of forking a sequence whose table holds an impossible page number: the new sequence is empty, and no count
changes for it."""
import pytest

from test_paged_gpu import lla  # noqa: F401
from test_paged_pages_gpu import Pair, ints, pools

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [-1, 20, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("at,pages", [(0, 1), (1, 3), (2, 3), (299, 300), (3, 300)])
def test_an_impossible_page_is_not_passed_on(lla, page, at, pages):  # noqa: F811
    pool = pools(20)
    rows = [[5] * pages, [6, 7]]
    P = Pair(lla, rows, [16 * pages - 3, 20], 301, pool)
    P.device.page_table[0, at] = page
    to = Pair(lla, [[], [], [], []], [9, 9, 9, 9], 301, pool)
    refs = ints([0] * 5 + [pages, 1, 1] + [0] * 12)
    lla.lla_paged_fork(P.device, to.device, ints([0, 1, -1, 0]), refs)
    assert lla.lla_stream_status() == 1
    assert to.device.lens.tolist() == [0, 20, 0, 0] and refs.tolist()[5:8] == [pages, 2, 2]
    assert to.device.page_table[1, :2].tolist() == [6, 7] and (to.device.page_table[[0, 2, 3]] == 0).all()
    # behind the length: not looked at
    P.device.page_table[0, at] = 5
    P.device.page_table[0, pages] = page
    lla.lla_paged_fork(P.device, to.device, ints([0, 1, -1, 0]), refs)
    assert lla.lla_stream_status() == 0 and to.device.lens.tolist() == [16 * pages - 3, 20, 0, 16 * pages - 3]
    assert refs.tolist()[5:8] == [3 * pages, 3, 3]
