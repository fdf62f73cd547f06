"""Float64 reference of the paged-cache operators on the CPU, written from the definitions, and the
error bounds that the kernels' arithmetic allows."""
import math

import torch

U32 = 2.0 ** -24  # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


class Problem:
    """A random paged cache with new tokens, on the CPU."""

    def __init__(self, lens, news, Hq=2, Hkv=1, d=64, dv=64, page=16, dtype=torch.bfloat16, probe=False,
                 seed=0, extra_pages=3, max_pages=None):
        g = torch.Generator().manual_seed(seed)
        self.lens_l, self.news_l = list(lens), list(news)
        self.Hq, self.Hkv, self.d, self.dv, self.page, self.dtype = Hq, Hkv, d, dv, page, dtype
        B = len(lens)
        counts = [-(-n // page) for n in lens]
        self.num_pages = sum(counts) + extra_pages
        order = torch.randperm(self.num_pages, generator=g).to(torch.int32)
        self.table = torch.zeros(B, max_pages or max(max(counts), 1), dtype=torch.int32)
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = order[at:at + c]
            at += c
        self.starts_l = [0]
        for t in news:
            self.starts_l.append(self.starts_l[-1] + t)
        N = self.starts_l[-1]
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.k = rnd(self.num_pages, Hkv, page, d).to(dtype)
        self.v = rnd(self.num_pages, Hkv, page, dv).to(dtype)
        self.q = rnd(N, Hq, d).to(dtype)
        self.r = (rnd(N, Hq, d) / math.sqrt(d)).to(dtype) if probe else None
        self.mass = torch.rand(self.num_pages, Hkv, page, generator=g)
        self.lens = torch.tensor(self.lens_l, dtype=torch.int32)
        self.starts = torch.tensor(self.starts_l, dtype=torch.int32)
        self.h = math.sqrt(d)

    def slots(self, b):
        j = torch.arange(self.lens_l[b])
        return self.table[b].long()[j // self.page], j % self.page

    def cuda(self, lla, mass=True):
        """(cache, q, r, starts) on the GPU."""
        cache = lla.PagedCache(self.k.cuda(), self.v.cuda(), self.table.cuda(), self.lens.cuda(),
                               self.mass.cuda() if mass else None)
        return cache, self.q.cuda(), None if self.r is None else self.r.cuda(), self.starts.cuda()


def attention(P, window=0, sinks=0, rounded_weights=True):
    """{out, lse, mass} in float64 and their bounds {out_tol, lse_tol, mass_tol}.

    Bounds, with u = 2^-24 and per row S = max_j sum_c |q_c k_jc| / h over its n visible keys:
    a logit is off by es = (d + 2) u S (twice that where the tensor cores' sums round towards zero),
    a weight relatively by 2 es + (n + 64) u (its own logit, the normaliser's terms, the n-term
    sum, the exponentials), a probe score by (d + 2) u sum_c |r_c k_jc|. The weights of bf16 inputs
    are rounded to bf16 once or, with a probe, twice (p and p t): half a step each. The output is
    rounded once."""
    N, g = P.q.shape[0], P.Hq // P.Hkv
    f = torch.float64
    out, lse = torch.zeros(N, P.Hq, P.dv, dtype=f), torch.full((N, P.Hq), -math.inf, dtype=f)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    mass, mass_tol = P.mass.to(f).clone(), torch.zeros(P.mass.shape, dtype=f)
    half = HALF[P.dtype]
    for b, (n, t) in enumerate(zip(P.lens_l, P.news_l)):
        if t == 0:
            continue
        pg, off = P.slots(b)
        j = torch.arange(n)
        pos = torch.arange(n - t, n)[:, None]
        seen = j[None] <= pos
        if window:
            seen &= (j[None] > pos - window) | (j[None] < sinks)
        a, e = P.starts_l[b], P.starts_l[b] + t
        for hk in range(P.Hkv):
            k, v = P.k[pg, hk, off].to(f), P.v[pg, hk, off].to(f)
            got, got_tol = torch.zeros(n, dtype=f), torch.zeros(n, dtype=f)
            for u in range(hk * g, hk * g + g):
                q = P.q[a:e, u].to(f)
                k0 = torch.where(seen.any(0)[:, None], k, torch.zeros_like(k))
                v0 = torch.where(seen.any(0)[:, None], v, torch.zeros_like(v))
                s = (q @ k0.T / P.h).masked_fill(~seen, -math.inf)
                S = torch.where(seen, q.abs() @ k0.abs().T / P.h, torch.zeros_like(s)).amax(-1, keepdim=True)
                some = seen.any(-1)
                m = torch.where(some[:, None], s.amax(-1, keepdim=True), torch.zeros(t, 1, dtype=f))
                w = torch.exp(s - m)
                tot = w.sum(-1, keepdim=True)
                p = torch.where(some[:, None], w / tot.clamp_min(1e-300), torch.zeros_like(w))
                es = 2 * (P.d + 2) * U32 * S
                rel = 2 * es + (seen.sum(-1, keepdim=True) + 64) * U32
                o = p @ v0
                A = p @ v0.abs()
                wtol = rel * A + (half if P.dtype != torch.float32 else 0.0) * A
                if P.r is not None:
                    r = P.r[a:e, u].to(f)
                    ts = torch.where(seen, r @ k0.T, torch.zeros_like(s))
                    te = 2 * (P.d + 2) * U32 * (r.abs() @ k0.abs().T)
                    tb = (p * ts).sum(-1, keepdim=True)
                    o = (p * (1 + tb - ts)) @ v0
                    A2 = (p * ts.abs()) @ v0.abs()
                    tb_abs = (p * ts.abs()).sum(-1, keepdim=True)
                    tb_err = (rel + rel) * tb_abs + (p * te).sum(-1, keepdim=True)
                    wtol = (rel + (half if P.dtype != torch.float32 else 0.0)) * ((1 + tb.abs()) * A + A2) \
                        + rel * A2 + (p * te) @ v0.abs() + tb_err * A
                out[a:e, u] = o
                out_tol[a:e, u] = wtol + half * (o.abs() + wtol) + 1e-30
                lse[a:e, u] = torch.where(some, (m + torch.log(tot.clamp_min(1e-300)))[:, 0],
                                          torch.full((t,), -math.inf, dtype=f))
                lse_tol[a:e, u] = (rel[:, 0] + 4 * U32 * m[:, 0].abs() + 16 * U32)
                got += p.sum(0)
                got_tol += (p * (2 * rel + 4 * U32 * m.abs() + 16 * U32)).sum(0)
            mass[pg, hk, off] += got
            mass_tol[pg, hk, off] += got_tol + (t * g + 8) * U32 * (got + P.mass[pg, hk, off].to(f))
    return {"out": out, "lse": lse, "mass": mass, "out_tol": out_tol, "lse_tol": lse_tol,
            "mass_tol": mass_tol}


def evict(P, budget, sinks, recent):
    """Kept positions [B][Hkv] as lists."""
    kept = []
    for b, n in enumerate(P.lens_l):
        pg, off = P.slots(b)
        row = []
        for hk in range(P.Hkv):
            mass = [(-math.inf, 1) if math.isnan(x) else (x, 0) for x in P.mass[pg, hk, off].tolist()]
            tail = max(sinks, n - recent)
            if n <= budget:
                row.append(list(range(n)))
                continue
            # larger first; NaN below everything, -infinity included; equal: the lower position
            order = sorted(range(sinks, tail), key=lambda j: (-mass[j][0], mass[j][1], j))
            row.append(sorted(list(range(sinks)) + order[:budget - sinks - recent] + list(range(n - recent, n))))
        kept.append(row)
    return kept
