"""GPU tests of keys whose logits are -infinity: they have no weight, whichever kernel adds the weights up,
and a row that sees no other key gives zero and -infinity as one that sees nothing."""
import math

import pytest
import torch

from paged_reference import HALF, U32, Problem
from test_paged_gpu import BF, F32, check, lla  # noqa: F401

pytestmark = pytest.mark.gpu


def without(P, seq, dead):
    """Softmax attention in float64 and its bounds (as paged_reference.attention derives them), where nobody
    sees position `dead` of sequence `seq`."""
    f, g, half = torch.float64, P.Hq // P.Hkv, HALF[P.dtype]
    N = P.q.shape[0]
    out, lse = torch.zeros(N, P.Hq, P.dv, dtype=f), torch.full((N, P.Hq), -math.inf, dtype=f)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    mass, mass_tol = P.mass.to(f).clone(), torch.zeros(P.mass.shape, dtype=f)
    for b, (n, t) in enumerate(zip(P.lens_l, P.news_l)):
        pg, off = P.slots(b)
        seen = torch.arange(n)[None] <= torch.arange(n - t, n)[:, None]
        if b == seq:
            seen[:, dead] = False
        rows, some = slice(P.starts_l[b], P.starts_l[b + 1]), seen.any(-1, keepdim=True)
        for u in range(P.Hq):
            hk = u // g
            q, k, v = P.q[rows, u].to(f), P.k[pg, hk, off].to(f), P.v[pg, hk, off].to(f)
            if b == seq:
                k[dead] = 0.0
            s = (q @ k.T / P.h).masked_fill(~seen, -math.inf)
            top = torch.where(some, s.amax(-1, keepdim=True), 0.0)
            tot = torch.exp(s - top).sum(-1, keepdim=True)
            p = torch.where(some, torch.exp(s - top) / tot.clamp_min(1e-300), 0.0)
            S = torch.where(seen, q.abs() @ k.abs().T / P.h, 0.0).amax(-1, keepdim=True)
            rel = 4 * (P.d + 2) * U32 * S + (seen.sum(-1, keepdim=True) + 64) * U32
            wtol = (rel + (half if P.dtype != F32 else 0.0)) * (p @ v.abs())
            out[rows, u] = p @ v
            out_tol[rows, u] = wtol + half * (out[rows, u].abs() + wtol) + 1e-30
            lse[rows, u] = torch.where(some, top + torch.log(tot.clamp_min(1e-300)), -math.inf)[:, 0]
            e = rel + 4 * U32 * top.abs() + 16 * U32
            lse_tol[rows, u] = e[:, 0]
            mass[pg, hk, off] += p.sum(0)
            mass_tol[pg, hk, off] += (p * (rel + e)).sum(0) + (t * g + 8) * U32 * (p.sum(0) + P.mass[pg, hk, off].to(f))
    return out, out_tol, lse, lse_tol, mass, mass_tol


@pytest.mark.parametrize("at", [0, 5, 150])
@pytest.mark.parametrize("lens,news", [([200], [1]), ([200, 9], [4, 2]), ([200], [200]), ([300, 400], [290, 90])])
@pytest.mark.parametrize("dtype,d,g,path", [(BF, 64, 4, 0), (BF, 64, 5, 0), (BF, 128, 3, 0), (BF, 64, 43, 0), (BF, 32, 2, 1),
                                            (F32, 64, 2, 0), (F32, 64, 20, 0), (F32, 128, 7, 0)])
def test_no_weight(lla, dtype, d, g, path, lens, news, at):  # noqa: F811
    P = Problem(lens, news, 2 * g, 2, d, d, 32, dtype, False, seed=91)
    P.q[..., 0] = P.q[..., 0].abs() + 0.5
    pg, off = P.slots(0)
    P.k[pg[at], :, off[at], 0] = -math.inf
    cache, q, r, starts = P.cuda(lla)
    out, lse = lla.lla_paged_attention(q, cache, starts, P.h, max_new=max(news), track_mass=True, path=path)
    assert lla.lla_stream_status() == 0
    want = without(P, 0, at)
    check("out", out, *want[:2])
    check("lse", lse, *want[2:4])
    check("mass", cache.mass, *want[4:])
