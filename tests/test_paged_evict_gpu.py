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
