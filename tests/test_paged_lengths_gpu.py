"""GPU tests of lengths that cannot be: the sequence is reported and left alone, and what its page table
holds beyond its pages (another sequence's, where a table is padded with any number) stays untouched."""
import pytest
import torch

from paged_reference import Problem, attention, evict
from test_paged_gpu import BF, F32, check, lla  # noqa: F401

pytestmark = pytest.mark.gpu


def broken(length, news, dtype=BF, d=64, g=2):
    """Two sequences; the first one's table ends in the second one's pages, its length is `length` beyond
    the table (or below zero)."""
    P = Problem([100, 400], news, g, 1, d, d, 16, dtype, True, seed=81)
    held = -(-100 // 16)
    P.table[0, held:] = P.table[1, :P.table.shape[1] - held]
    P.lens[0] = length if length < 0 else P.table.shape[1] * P.page + length
    return P


LENGTHS = [-1, -2**31, 1, 100, 2**30]


@pytest.mark.parametrize("length", LENGTHS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_append(lla, dtype, length):  # noqa: F811
    P = broken(length, [20, 3], dtype)
    cache, _, _, starts = P.cuda(lla)
    k, v = (torch.randn(23, 1, 64).to(dtype) for _ in range(2))
    lla.lla_paged_append(k.cuda(), v.cuda(), cache, starts)
    assert lla.lla_stream_status() == 1
    pg, off = (x[-3:] for x in P.slots(1))
    P.k[pg, 0, off], P.v[pg, 0, off], P.mass[pg, 0, off] = k[20:, 0], v[20:, 0], 0.0
    assert torch.equal(cache.k_pages.cpu(), P.k) and torch.equal(cache.v_pages.cpu(), P.v)
    assert torch.equal(cache.mass.cpu(), P.mass)


@pytest.mark.parametrize("length", LENGTHS)
@pytest.mark.parametrize("news", [[1, 1], [3, 2], [60, 70]])
@pytest.mark.parametrize("dtype,d,g,path", [(BF, 64, 2, 0), (BF, 128, 3, 0), (BF, 64, 4, 1), (F32, 64, 2, 0), (F32, 128, 20, 0)])
def test_attention(lla, dtype, d, g, path, news, length):  # noqa: F811
    P = broken(length, news, dtype, d, g)
    cache, q, r, starts = P.cuda(lla)
    out, lse = lla.lla_paged_attention(q, cache, starts, P.h, r=r, max_new=max(news), track_mass=True, path=path)
    assert lla.lla_stream_status() == 1
    clean = Problem([100, 400], news, g, 1, d, d, 16, dtype, True, seed=81)
    ref, (pg, off) = attention(clean), clean.slots(1)
    rows = slice(news[0], None)
    check("out", out[rows], ref["out"][rows], ref["out_tol"][rows])
    check("lse", lse[rows], ref["lse"][rows], ref["lse_tol"][rows])
    check("mass", cache.mass.cpu()[pg, :, off], ref["mass"][pg, :, off], ref["mass_tol"][pg, :, off])
    rest = torch.ones(P.num_pages, dtype=torch.bool)
    rest[P.table[1].long()] = False
    assert torch.equal(cache.mass.cpu()[rest], clean.mass[rest])


@pytest.mark.parametrize("length", LENGTHS)
def test_evict(lla, length):  # noqa: F811
    P = broken(length, [0, 0], F32, 16)
    cache, _, _, _ = P.cuda(lla)
    pages = [[0, 1, 2, 3], [1, 2, 3, 4]]  # room for 60 positions; the first sequence needs none
    to = lla.PagedCache(torch.zeros(5, 1, 16, 16, device="cuda"), torch.zeros(5, 1, 16, 16, device="cuda"),
                        torch.tensor(pages, dtype=torch.int32, device="cuda"),
                        torch.full((2,), 7, dtype=torch.int32, device="cuda"), torch.zeros(5, 1, 16, device="cuda"))
    kept = lla.lla_paged_evict(cache, to, 60, sinks=2, recent=9).cpu()
    assert lla.lla_stream_status() == 1
    P.lens_l[0] = 0
    ref = evict(P, 60, 2, 9)
    assert kept[1, 0].tolist() == ref[1][0] and to.lens[1] == 60 and to.lens[0] == 0
    assert (kept[0, 0] == -1).all() and (to.k_pages[0] == 0).all()
    pg, off = P.slots(1)
    i = torch.arange(60)
    at = torch.tensor(pages[1])[i // 16], i % 16
    assert torch.equal(to.k_pages.cpu()[at[0], 0, at[1]], P.k[pg[ref[1][0]], 0, off[ref[1][0]]])
