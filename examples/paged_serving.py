"""Serving with a paged cache: prompts in chunks, decode steps that track the attention weights, and
eviction when a sequence outgrows its share of the pages.

    python examples/paged_serving.py

One Parallax attention layer over random projections (a stand-in for a model's q, k, v and probe):
three sequences bring their prompts in chunks of different sizes, next to each other in one batch,
then decode token by token. Sequences that pass `limit` positions are cut back to `budget`: the
first tokens, the most recent ones, and those that received the most attention. Without eviction
the outputs are the contiguous operators': the prompts' are compared with lla_parallax_forward.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import local_linear_attention_gb300 as lla  # noqa: E402


class Pages:
    """Pages of one layer's cache and which are free; the tables live on the device."""

    def __init__(self, num_pages, kv_heads, page, d, max_seqs, max_pages, device="cuda"):
        bf = dict(dtype=torch.bfloat16, device=device)
        self.k = torch.empty(num_pages, kv_heads, page, d, **bf)
        self.v = torch.empty(num_pages, kv_heads, page, d, **bf)
        self.mass = torch.zeros(num_pages, kv_heads, page, device=device)
        self.page, self.free = page, list(range(num_pages))[::-1]
        self.held = [[] for _ in range(max_seqs)]
        self.len = [0] * max_seqs
        self.max_pages, self.device = max_pages, device

    def grow(self, seq, tokens):
        """Pages for `tokens` more positions of a sequence."""
        self.len[seq] += tokens
        while len(self.held[seq]) * self.page < self.len[seq]:
            self.held[seq].append(self.free.pop())

    def table(self, held=None):
        rows = [h + [0] * (self.max_pages - len(h)) for h in (held or self.held)]
        return torch.tensor(rows, dtype=torch.int32, device=self.device)

    def cache(self):
        lens = torch.tensor(self.len, dtype=torch.int32, device=self.device)
        return lla.PagedCache(self.k, self.v, self.table(), lens, self.mass)

    def evict(self, seqs, budget, sinks, recent):
        """Cuts the sequences back to `budget` positions, in fresh pages; the old ones are free then.
        The others keep theirs: they go through as empty."""
        fresh = [[self.free.pop() for _ in range(-(-min(self.len[s], budget) // self.page))] if s in seqs else []
                 for s in range(len(self.len))]
        source = lla.PagedCache(self.k, self.v, self.table(), torch.tensor(
            [n if s in seqs else 0 for s, n in enumerate(self.len)], dtype=torch.int32, device=self.device), self.mass)
        dest = lla.PagedCache(self.k, self.v, self.table(fresh), torch.zeros_like(source.lens), self.mass)
        kept = lla.lla_paged_evict(source, dest, budget, sinks=sinks, recent=recent)
        for s in seqs:
            self.free += self.held[s]
            self.held[s], self.len[s] = fresh[s], min(self.len[s], budget)
        return kept


def step(pages, q, k, v, r, news, h, track):
    """Appends the new tokens of all sequences (news[s] each) and attends."""
    for s, n in enumerate(news):
        pages.grow(s, n)
    starts = torch.tensor([0] + torch.tensor(news).cumsum(0).tolist(), dtype=torch.int32, device=q.device)
    cache = pages.cache()
    lla.lla_paged_append(k, v, cache, starts)
    return lla.lla_paged_attention(q, cache, starts, h, r=r, max_new=max(news), track_mass=track)


def serve(prompts=(700, 90, 300), chunk=256, decode=40, limit=512, budget=384, q_heads=8, kv_heads=2, d=64,
          page=32, seed=0):
    """Runs the example; returns (worst difference of the prompts' outputs from the contiguous forward,
    lengths at the end)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda n, heads, scale=1.0: (torch.randn(n, heads, d, generator=g, device="cuda") * scale).bfloat16()  # noqa: E731
    h, B = math.sqrt(d), len(prompts)
    pages = Pages(4 * sum(-(-n // page) + 4 for n in prompts), kv_heads, page, d, B, -(-max(prompts) // page) + 4)
    data = [(rnd(n, q_heads), rnd(n, kv_heads), rnd(n, kv_heads), rnd(n, q_heads, d ** -0.5)) for n in prompts]

    # The prompts, a chunk of each per step until all are in.
    outs, done = [[] for _ in prompts], [0] * B
    while any(x < n for x, n in zip(done, prompts)):
        news = [min(chunk, n - x) for x, n in zip(done, prompts)]
        batch = [torch.cat([t[x:x + c] for t, x, c in zip(parts, done, news)]) for parts in zip(*data)]
        out, _ = step(pages, *batch, news, h, track=True)
        for s, o in enumerate(out.split(news)):
            outs[s].append(o)
            done[s] += news[s]
    worst = 0.0
    for s, (q, k, v, r) in enumerate(data):
        group = q_heads // kv_heads
        heads = lambda x: x.transpose(0, 1)[None].contiguous()  # noqa: E731
        full = lla.lla_parallax_forward(heads(q), heads(k.repeat_interleave(group, 1)),
                                        heads(v.repeat_interleave(group, 1)), heads(r), h)
        mine = heads(torch.cat(outs[s]))
        worst = max(worst, float((mine - full).float().norm() / full.float().norm()))

    # Decode; whoever passes the limit is cut back.
    for _ in range(decode):
        step(pages, rnd(B, q_heads), rnd(B, kv_heads), rnd(B, kv_heads), rnd(B, q_heads, d ** -0.5), [1] * B, h, track=True)
        over = [s for s in range(B) if pages.len[s] > limit]
        if over:
            kept = pages.evict(over, budget, sinks=4, recent=64)
            for s in over:
                pos = kept[s, 0][kept[s, 0] >= 0]
                assert pos.numel() == budget and bool((pos[1:] > pos[:-1]).all())
    torch.cuda.synchronize()
    if lla.lla_stream_status() != 0:
        raise RuntimeError("liblla reported an error")
    return worst, list(pages.len)


if __name__ == "__main__":
    difference, lengths = serve()
    print(f"prompts: relative difference from the contiguous forward {difference:.1e}; lengths at the end {lengths}")
