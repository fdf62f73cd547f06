"""GPU tests of token buffers that are longer than what the sequences take of them, as buffers of a fixed
size are: starts that begin above zero and end below the buffer's end."""
import math

import pytest
import torch

from paged_reference import Problem, attention
from test_paged_gpu import BF, F32, check, lla  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("before,behind", [(3, 0), (0, 5), (7, 300)])
@pytest.mark.parametrize("lens,news", [([100, 30], [1, 1]), ([90, 300, 5], [4, 2, 5]), ([200, 300], [130, 1])])
@pytest.mark.parametrize("dtype,d,Hq,Hkv,probe,path", [(BF, 64, 4, 2, True, 0), (BF, 128, 5, 1, False, 0), (BF, 128, 4, 4, True, 0),
                                                       (BF, 64, 2, 2, True, 1), (F32, 64, 4, 2, True, 0), (F32, 32, 20, 1, False, 0)])
def test_rows_that_no_sequence_covers(lla, dtype, d, Hq, Hkv, probe, path, lens, news, before, behind):  # noqa: F811
    """They take no part (they hold NaN) and their outputs are not written."""
    P = Problem(lens, news, Hq, Hkv, d, d, 16, dtype, probe, seed=111)
    cache, q, r, starts = P.cuda(lla)
    junk = lambda n, x: torch.full((n, *x.shape[1:]), math.nan, dtype=x.dtype, device="cuda")  # noqa: E731
    around = lambda x: None if x is None else torch.cat([junk(before, x), x, junk(behind, x)])  # noqa: E731
    q2, r2, starts2 = around(q), around(r), starts + before
    out, lse = torch.full_like(q2, 7.0), torch.full(q2.shape[:2], 7.0, device="cuda")
    lla.lla_paged_attention(q2, cache, starts2, P.h, r=r2, max_new=max(news), track_mass=True, out=out, lse=lse, path=path)
    assert lla.lla_stream_status() == 0
    rows, ref = slice(before, before + q.shape[0]), attention(P)
    check("out", out[rows], ref["out"], ref["out_tol"])
    check("lse", lse[rows], ref["lse"], ref["lse_tol"])
    check("mass", cache.mass, ref["mass"], ref["mass_tol"])
    rest = torch.ones(q2.shape[0], dtype=torch.bool)
    rest[rows] = False
    assert (out.cpu()[rest] == 7).all() and (lse.cpu()[rest] == 7).all()
    k, v = (torch.randn(q.shape[0], Hkv, d).to(dtype).cuda() for _ in range(2))
    lla.lla_paged_append(around(k), around(v), cache, starts2)
    assert lla.lla_stream_status() == 0
    for b, (n, t) in enumerate(zip(lens, news)):
        pg, off = (x[-t:] for x in P.slots(b))
        P.k[pg, :, off], P.v[pg, :, off] = (x[P.starts_l[b]:P.starts_l[b + 1]].cpu() for x in (k, v))
    assert torch.equal(cache.k_pages.cpu(), P.k) and torch.equal(cache.v_pages.cpu(), P.v)
