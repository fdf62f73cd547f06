"""GPU tests of eviction from sequences so long that eight blocks select for a head."""
import pytest
import torch

from paged_reference import Problem
from test_paged_gpu import F32, lla, run_evict  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,heads", [(40011, 1), (65536, 2)])
def test_selection_over_a_cluster_of_eight(lla, n, heads):  # noqa: F811
    """One long sequence, a cluster of eight blocks a head; whole stretches of equal weights, so that ties
    run over the blocks' borders."""
    P = Problem([n], [0], heads, heads, 16, 16, 64, F32, seed=101)
    g = torch.Generator().manual_seed(3)
    levels = torch.tensor([0.25, 0.5, 0.5, 0.5, 2.0])
    P.mass = levels[torch.randint(0, 5, P.mass.shape, generator=g)]
    pg, off = P.slots(0)
    P.mass[pg[9000:21000], :, off[9000:21000]] = 0.5
    for budget in (n // 4, n // 2, n - 100):
        run_evict(lla, P, budget, 16, 100)


def test_tables_without_pages(lla):  # noqa: F811
    """Sequences that hold nothing yet, in tables of no columns: nothing is kept."""
    from test_paged_abi import cache
    import ctypes
    keep = [torch.zeros(64, dtype=torch.int32, device="cuda") for _ in range(5)]
    keep[2].fill_(9)
    at = [x.data_ptr() for x in keep]
    f = dict(k_pages=at[0], v_pages=at[0], mass=at[0], num_seqs=2, kv_heads=2, max_pages=0, num_pages=0)
    a, b = cache(lla, **f, page_table=at[1], lens=at[1]), cache(lla, **f, page_table=at[4], lens=at[2])
    assert lla._load().lla_paged_evict(ctypes.byref(a), ctypes.byref(b), 3, 1, 1, at[3], None) == 0
    assert lla.lla_stream_status() == 0
    assert keep[3][:12].tolist() == [-1] * 12 and keep[2][:3].tolist() == [0, 0, 9]
