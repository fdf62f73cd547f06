"""GPU tests of Parallax attention over a paged cache where the probe scores t = r.k have a large mean, or
follow the logits: the output depends on their differences only, and so must its error."""
import math

import pytest
import torch

from paged_reference import HALF, U32, Problem, attention
from test_paged_gpu import BF, F32, check, lla  # noqa: F401

pytestmark = pytest.mark.gpu


def offset(P, mean, follow=0.0, scale=1.0, seed=0):
    """Keys with a common offset along which the probe scores have about this mean; probes that lie along
    their queries by `follow`, queries scaled."""
    u = torch.randn(P.d, generator=torch.Generator().manual_seed(seed))
    u = u / u.norm() * abs(mean)
    q = (P.q.float() * scale).to(P.dtype)
    P.k = (P.k.float() + u).to(P.dtype)
    P.r = (P.r.float() + follow * q.float() / math.sqrt(P.d) + (u / mean if mean else 0.0)).to(P.dtype)
    P.q = q
    return P


def bound(P, window=0, sinks=0):
    """(out, tolerance) in float64. With o = v~ - C, v~ = sum p v, C = sum p (t - t~) (v - v~), a weight off by
    the relative d_j moves o by sum p_j d_j ((v_j - v~) (1 - (t_j - t~)) + C): d_j is a weight's
    rounding to bf16 (half a step) and what its logit and exponential are off by (see `attention`), a few
    times over for the terms of second order. p t is held to a bf16 pair (half a step of half a step), and
    the fp32 sums of p v and p t v, over whose difference o is taken, are off by (n + 64) u of their terms."""
    f, g = torch.float64, P.Hq // P.Hkv
    half = HALF[P.dtype] if P.dtype != F32 else 0.0
    out = torch.zeros(P.q.shape[0], P.Hq, P.dv, dtype=f)
    tol = torch.zeros_like(out)
    for b, (n, t) in enumerate(zip(P.lens_l, P.news_l)):
        pg, off = P.slots(b)
        j, pos = torch.arange(n), torch.arange(n - t, n)[:, None]
        seen = j[None] <= pos
        if window:
            seen &= (j[None] > pos - window) | (j[None] < sinks)
        rows = slice(P.starts_l[b], P.starts_l[b + 1])
        for u in range(P.Hq):
            k, v = P.k[pg, u // g, off].to(f), P.v[pg, u // g, off].to(f)
            q, r = P.q[rows, u].to(f), P.r[rows, u].to(f)
            s = (q @ k.T / P.h).masked_fill(~seen, -math.inf)
            p = torch.softmax(s, -1)
            S = torch.where(seen, q.abs() @ k.abs().T / P.h, 0.0).amax(-1, keepdim=True)
            rel = 4 * (P.d + 2) * U32 * S + (seen.sum(-1, keepdim=True) + 64) * U32
            ts, te = r @ k.T, 2 * (P.d + 2) * U32 * (r.abs() @ k.abs().T)
            tb = (p * ts).sum(-1, keepdim=True)
            mean = p @ v
            c = (p * (ts - tb)) @ v
            dev = v[None] - mean[:, None]                                  # [rows, keys, dv]
            grad = (dev * (1 - (ts - tb))[..., None] + c[:, None]).abs()
            e = (p[..., None] * grad).sum(1) * (half + rel) * (1 + 8 * half)
            e += ((p * te)[..., None] * dev.abs()).sum(1)
            A, A2 = p @ v.abs(), (p * ts.abs()) @ v.abs()
            A2t = A2 + (p * ts.abs()).sum(-1, keepdim=True) * A
            e += (seen.sum(-1, keepdim=True) + 64) * U32 * (A + A2t) + half * half * A2t
            o = mean - c
            out[rows, u] = o
            tol[rows, u] = e + HALF[P.dtype] * (o.abs() + e) + 1e-30
    return out, tol


MEANS = [(0.0, 0.0, 1.0), (2.5, 0.0, 1.0), (-25.0, 0.0, 1.0), (25.0, 1.0, 3.0)]


@pytest.mark.parametrize("mean,follow,scale", MEANS)
@pytest.mark.parametrize("lens,news", [([40, 700, 1], [1, 1, 1]), ([300, 90], [6, 2]), ([700, 130, 50], [300, 130, 1])])
@pytest.mark.parametrize("dtype,d,dv,Hq,Hkv", [(BF, 64, 64, 4, 4), (BF, 128, 128, 4, 2), (BF, 64, 32, 6, 2),
                                               (BF, 128, 64, 10, 1), (F32, 64, 64, 4, 2)])
def test_scores_with_a_large_mean(lla, dtype, d, dv, Hq, Hkv, lens, news, mean, follow, scale):  # noqa: F811
    P = offset(Problem(lens, news, Hq, Hkv, d, dv, 32, dtype, True, seed=41), mean, follow, scale)
    cache, q, r, starts = P.cuda(lla)
    for window, sinks in ((0, 0), (60, 5)):
        out, lse = lla.lla_paged_attention(q, cache, starts, P.h, r=r, max_new=max(news), window=window, sinks=sinks)
        assert lla.lla_stream_status() == 0
        check("out", out, *bound(P, window, sinks))
        ref = attention(P, window, sinks)
        check("lse", lse, ref["lse"], ref["lse_tol"])


@pytest.mark.parametrize("mean", [2.5, 25.0])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("news", [1, 70])
def test_parts_of_long_sequences(lla, d, news, mean):  # noqa: F811
    """Partial results joined in a cluster, through scratch, and of a tile that was cut."""
    for lens in ([3001, 2048], [30001]):
        P = offset(Problem(lens, [news] * len(lens), 2, 1, d, d, 64, BF, True, seed=42), mean)
        cache, q, r, starts = P.cuda(lla)
        out, _ = lla.lla_paged_attention(q, cache, starts, P.h, r=r, max_new=news)
        assert lla.lla_stream_status() == 0
        check("out", out, *bound(P))


@pytest.mark.parametrize("mean,follow,scale", MEANS)
def test_as_near_as_the_contiguous_forward(lla, mean, follow, scale):  # noqa: F811
    """Both round each weight and each output once: the same error, up to the roundings' chance (a quarter)."""
    T, H, d = 400, 4, 64
    P = offset(Problem([T, T], [T, T], H, H, d, d, 16, BF, True, seed=43), mean, follow, scale)
    cache, q, r, starts = P.cuda(lla)
    ref = bound(P)[0]
    out, _ = lla.lla_paged_attention(q, cache, starts, P.h, r=r, max_new=T)
    k = torch.stack([P.k[P.slots(b)[0], :, P.slots(b)[1]] for b in range(2)]).transpose(1, 2).contiguous().cuda()
    v = torch.stack([P.v[P.slots(b)[0], :, P.slots(b)[1]] for b in range(2)]).transpose(1, 2).contiguous().cuda()
    heads = lambda x: x.reshape(2, T, H, d).transpose(1, 2).contiguous()  # noqa: E731
    full = lla.lla_parallax_forward(heads(q), k, v, heads(r), P.h)
    ours = (heads(out).cpu().double() - heads(ref)).norm() / ref.norm()
    theirs = (full.cpu().double() - heads(ref)).norm() / ref.norm()
    assert ours <= 1.25 * theirs, (float(ours), float(theirs))
