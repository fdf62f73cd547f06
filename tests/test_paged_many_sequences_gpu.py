"""GPU tests of drafting operators over more sequences than their kernels keep in shared memory (1024 for the rotated
append, 2048 for trees on the tensor cores), many of them without new tokens. References and bounds as in
test_rotary_gpu.py and test_paged_tree_gpu.py."""
import random

import pytest
import torch

from paged_reference import Problem
from paged_tree_reference import attention, trees
from test_paged_gpu import BF, F32, check, lla  # noqa: F401
from test_paged_tree_gpu import flat
from test_rotary_gpu import turned

pytestmark = pytest.mark.gpu


def batch(B, most, seed):
    rng = random.Random(seed)
    news = [rng.choice([0, 0, 1, rng.randint(0, most)]) for _ in range(B)]
    return [t + rng.randint(0, 40) for t in news], news


@pytest.mark.parametrize("before", [0, 7])
@pytest.mark.parametrize("dtype,B", [(BF, 1023), (F32, 1024), (BF, 1025), (BF, 3000)])
def test_append(lla, dtype, B, before):  # noqa: F811
    """Rows before the first sequence's and behind the last one's stay as they are."""
    lens, news = batch(B, 5, B)
    P = Problem(lens, news, 3, 1, 32, 16, 16, dtype, True, seed=1)
    N = sum(news)
    g = torch.Generator().manual_seed(2)
    rows = before + N + 4
    k, v = torch.randn(rows, 1, 32, generator=g).to(dtype), torch.randn(rows, 1, 16, generator=g).to(dtype)
    q, r = torch.randn(rows, 3, 32, generator=g).to(dtype), torch.randn(rows, 3, 32, generator=g).to(dtype)
    cache, _, _, starts = P.cuda(lla)
    spec = lla.RotarySpec(20, base=300.0)
    out_q, out_r = torch.full_like(q, 7).cuda(), torch.full_like(q, 7).cuda()
    lla.lla_paged_append_rotary(k.cuda(), v.cuda(), cache, starts + before, spec, q.cuda(), r.cuda(), q_out=out_q, r_out=out_r)
    assert lla.lla_stream_status() == 0
    where = [(b, n - t + i) for b, (n, t) in enumerate(zip(lens, news)) for i in range(t)]
    pos = torch.tensor([j for _, j in where])[:, None]
    mine = slice(before, before + N)
    for x, y in ((q, out_q), (r, out_r)):
        check("out", y[mine], *turned(x[mine], spec, pos))
        assert (y[:before] == 7).all() and (y[before + N:] == 7).all()
    pg = torch.tensor([int(P.table[b, j // 16]) for b, j in where])
    off = torch.tensor([j % 16 for _, j in where])
    check("k", cache.k_pages.cpu()[pg, :, off], *turned(k[mine], spec, pos))
    assert torch.equal(cache.v_pages.cpu()[pg, :, off], v[mine])
    rest = torch.ones(P.num_pages, 16, dtype=torch.bool)
    rest[pg, off] = False
    assert torch.equal(cache.k_pages.cpu().transpose(1, 2)[rest], P.k.transpose(1, 2)[rest])


@pytest.mark.parametrize("dtype,B,wide", [(BF, 2048, 90), (BF, 2049, 90), (BF, 2500, 12), (F32, 2500, 90)])
def test_trees(lla, dtype, B, wide):  # noqa: F811
    lens, news = batch(B, 3, B)
    news[B // 2] = wide
    lens[B // 2] = wide + 30
    P = Problem(lens, news, 2, 1, 64, 64, 16, dtype, True, seed=3)
    forest = trees(news, 2)
    ref = attention(P, forest, window=25, sinks=2)
    cache, q, r, starts = P.cuda(lla, mass=False)
    out, lse = lla.lla_paged_tree_attention(q, cache, starts, flat(forest), P.h, r=r, max_new=wide, window=25, sinks=2)
    assert lla.lla_stream_status() == 0
    check("out", out, ref["out"], ref["out_tol"])
    check("lse", lse, ref["lse"], ref["lse_tol"])
