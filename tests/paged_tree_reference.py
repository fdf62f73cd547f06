"""Float64 reference of attention of drafted trees over a paged cache, on the CPU, and the error bounds
that the kernels' arithmetic allows (those of paged_reference.attention)."""
import math
import random

import torch

from paged_reference import HALF, U32


def trees(news, branch, seed=0):
    """A forest for each number of nodes: branch 1 is near a chain, more is wider; 0 is a chain, -1 all roots."""
    rng = random.Random(seed)
    out = []
    for t in news:
        if branch == 0:
            out.append([i - 1 for i in range(t)])
        elif branch < 0:
            out.append([-1] * t)
        else:
            out.append([rng.randint(max(-1, i // branch - 3), i - 1) if rng.random() < 0.3 else
                        max(-1, min(i - 1, i // branch - 1)) for i in range(t)])
    return out


def depths(tree):
    d = []
    for a in tree:
        d.append(0 if a < 0 else d[a] + 1)
    return d


def sight(n, tree, window, sinks):
    """Which of n positions each node sees: [nodes, n]."""
    t = len(tree)
    first, d = n - t, depths(tree)
    seen = torch.zeros(t, n, dtype=torch.bool)
    for i in range(t):
        pos, line, a = first + d[i], {i}, tree[i]
        while a >= 0:
            line.add(a)
            a = tree[a]
        for j in range(n):
            at = j if j < first else first + d[j - first]
            if (j < first or j - first in line) and (not window or at > pos - window or at < sinks):
                seen[i, j] = True
    return seen


def attention(P, forest, window=0, sinks=0):
    """{out, lse} in float64 and their bounds {out_tol, lse_tol}: see paged_reference.attention."""
    N, g = P.q.shape[0], P.Hq // P.Hkv
    f = torch.float64
    out, lse = torch.zeros(N, P.Hq, P.dv, dtype=f), torch.full((N, P.Hq), -math.inf, dtype=f)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    half = HALF[P.dtype]
    rounded = half if P.dtype != torch.float32 else 0.0
    for b, (n, t) in enumerate(zip(P.lens_l, P.news_l)):
        if t == 0:
            continue
        pg, off = P.slots(b)
        seen = sight(n, forest[b], window, sinks)
        a, e = P.starts_l[b], P.starts_l[b] + t
        for u in range(P.Hq):
            k, v = P.k[pg, u // g, off].to(f), P.v[pg, u // g, off].to(f)
            anyone = seen.any(0)[:, None]
            k, v = torch.where(anyone, k, torch.zeros_like(k)), torch.where(anyone, v, torch.zeros_like(v))
            q = P.q[a:e, u].to(f)
            s = (q @ k.T / P.h).masked_fill(~seen, -math.inf)
            S = torch.where(seen, q.abs() @ k.abs().T / P.h, torch.zeros_like(s)).amax(-1, keepdim=True)
            m = s.amax(-1, keepdim=True)
            w = torch.exp(s - m)
            tot = w.sum(-1, keepdim=True)
            p = w / tot
            rel = 4 * (P.d + 2) * U32 * S + (seen.sum(-1, keepdim=True) + 64) * U32
            o, A = p @ v, p @ v.abs()
            tol = (rel + rounded) * A
            if P.r is not None:
                r = P.r[a:e, u].to(f)
                ts = torch.where(seen, r @ k.T, torch.zeros_like(s))
                te = 2 * (P.d + 2) * U32 * (r.abs() @ k.abs().T)
                tb, tb_abs = (p * ts).sum(-1, keepdim=True), (p * ts.abs()).sum(-1, keepdim=True)
                o = (p * (1 + tb - ts)) @ v
                A2 = (p * ts.abs()) @ v.abs()
                tb_err = 2 * rel * tb_abs + (p * te).sum(-1, keepdim=True)
                tol = (rel + rounded) * ((1 + tb.abs()) * A + A2) + rel * A2 + (p * te) @ v.abs() + tb_err * A
            out[a:e, u] = o
            out_tol[a:e, u] = tol + half * (o.abs() + tol) + 1e-30
            lse[a:e, u] = (m + torch.log(tot))[:, 0]
            lse_tol[a:e, u] = rel[:, 0] + 4 * U32 * m[:, 0].abs() + 16 * U32
    return {"out": out, "lse": lse, "out_tol": out_tol, "lse_tol": lse_tol}
