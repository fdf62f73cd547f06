"""GPU tests of weight tracking where the page table has room for so many positions that the attention does
not keep its logits: the weights are computed again from q and k."""
import pytest

from paged_reference import Problem
from test_paged_gpu import BF, F32, lla, run_and_check  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 7)])
@pytest.mark.parametrize("lens,news", [([1500, 40], [1, 1]), ([900, 1], [40, 1])])
@pytest.mark.parametrize("dtype,d,Hkv,g,probe", [(BF, 64, 2, 16, False), (BF, 128, 4, 8, True), (BF, 32, 2, 5, False),
                                                 (F32, 64, 2, 16, False), (F32, 64, 2, 16, True)])
def test_wide_tables(lla, dtype, d, Hkv, g, probe, lens, news, window, sinks):  # noqa: F811
    rows = min(max(news) * g, 16 if dtype == F32 else 8 if probe else 16)
    pages = (1 << 31) // (4 * rows * 2 * Hkv * 1024) + 2   # past two gibibytes of logits for 2 sequences
    P = Problem(lens, news, Hkv * g, Hkv, d, d, 1024, dtype, probe, seed=61, max_pages=pages)
    run_and_check(lla, P, window, sinks)
    cache, q, r, starts = P.cuda(lla)
    kw = dict(r=r, max_new=max(news), window=window, sinks=sinks)
    extra = lla.lla_paged_workspace_size(q, cache, starts, P.h, track_mass=True, **kw) - \
        lla.lla_paged_workspace_size(q, cache, starts, P.h, **kw)
    assert extra <= 1 << 31
    if not window:
        assert extra < 1 << 20
