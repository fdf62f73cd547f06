"""GPU tests of the tensor-core attention where a row's reference grows in many steps: the products of a
step may only start once all of the row's accumulators have been rescaled, by whichever warps do it."""
import pytest
import torch

from paged_reference import Problem
from test_paged_gpu import BF, lla, run_and_check  # noqa: F401

pytestmark = pytest.mark.gpu


def staircase(P, nats, tile=128):
    """Keys of one direction whose logits are about `nats` higher in each tile than in the one before,
    and queries that lie along it."""
    for b, n in enumerate(P.lens_l):
        pg, off = P.slots(b)
        for hk in range(P.Hkv):
            u = P.k[pg[0], hk, off[0]].float()
            u = u / u.norm() * P.h
            level = (torch.arange(n) // tile).float() * nats / P.h
            P.k[pg, hk, off] = (P.k[pg, hk, off].float() * 0.2 + level[:, None] * u[None]).to(P.dtype)
            g = P.Hq // P.Hkv
            P.q[P.starts_l[b]:P.starts_l[b + 1], hk * g:hk * g + g] += u.to(P.dtype)
    return P


@pytest.mark.parametrize("window,sinks", [(0, 0), (1500, 40)])
@pytest.mark.parametrize("nats", [0.8, 1.4, 6.0])
@pytest.mark.parametrize("d,dv", [(128, 128), (128, 64), (64, 128), (64, 64)])
def test_references_that_grow_in_many_steps(lla, d, dv, nats, window, sinks):  # noqa: F811
    P = staircase(Problem([3000, 2100], [300, 260], 4, 2, d, dv, 64, BF, True, seed=31), nats)
    first = None
    for _ in range(4):
        now = run_and_check(lla, P, window, sinks, track=False)[:2]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
        first = now
