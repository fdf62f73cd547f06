"""GPU tests of a sequence that brings more new tokens than the call says: it is reported where its rows
were not computed, and the other sequences' outputs and weights are as they are without it."""
import pytest
import torch

from paged_reference import Problem, attention
from test_paged_gpu import BF, F32, check, lla  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,news,long", [([90, 40, 33, 70], [60, 1, 2, 3], 0), ([700, 40, 333, 70], [1, 300, 20, 17], 1),
                                            ([50, 60, 300, 9], [4, 4, 1, 9], 3), ([900, 60, 800, 77], [1, 4, 400, 1], 2)])
@pytest.mark.parametrize("dtype,d,Hq,Hkv,probe", [(F32, 64, 4, 2, True), (F32, 128, 17, 1, False), (F32, 32, 3, 3, False),
                                                  (BF, 64, 4, 2, True), (BF, 128, 5, 1, False)])
def test_the_others_are_right(lla, dtype, d, Hq, Hkv, probe, lens, news, long):  # noqa: F811
    P = Problem(lens, news, Hq, Hkv, d, d, 16, dtype, probe, seed=71)
    others = [b for b in range(4) if b != long]
    cache, q, r, starts = P.cuda(lla)
    out, lse = lla.lla_paged_attention(q, cache, starts, P.h, r=r, max_new=max(news[b] for b in others), track_mass=True)
    status = lla.lla_stream_status()
    assert status in ((1,) if dtype == F32 else (0, 1))
    ref = attention(P)
    for b in others:
        rows = slice(P.starts_l[b], P.starts_l[b + 1])
        check("out", out[rows], ref["out"][rows], ref["out_tol"][rows])
        check("lse", lse[rows], ref["lse"][rows], ref["lse_tol"][rows])
        pg, off = P.slots(b)
        check("mass", cache.mass.cpu()[pg, :, off], ref["mass"][pg, :, off], ref["mass_tol"][pg, :, off])
    again, _ = lla.lla_paged_attention(q, cache, starts, P.h, r=r, max_new=max(news))
    assert lla.lla_stream_status() == 0
    check("out", again, ref["out"], ref["out_tol"])


def test_a_sequence_far_down_the_list_is_reported(lla):  # noqa: F811
    news = [1] * 700
    news[650] = 40
    P = Problem([50] * 700, news, 2, 2, 16, 16, 16, F32, False, seed=72)
    cache, q, r, starts = P.cuda(lla)
    out, _ = lla.lla_paged_attention(q, cache, starts, P.h, max_new=1)
    assert lla.lla_stream_status() == 1
    ref = attention(P)
    keep = torch.ones(q.shape[0], dtype=torch.bool)
    keep[650:690] = False
    check("out", out.cpu()[keep], ref["out"][keep], ref["out_tol"][keep])
