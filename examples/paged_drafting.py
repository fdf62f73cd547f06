"""Drafted decoding on a paged cache: samples forked from one prompt, trees of drafted tokens verified in one
pass, the accepted path kept.

    python examples/paged_drafting.py

A toy model (random weights, full precision, Parallax attention with rotary positions, a table of pages that its layers
share) decodes greedily, token by token and again with drafts. The drafts are the first run's tokens
with mistakes, in place of a draft model's: a tree holds a stretch of them and false turns beside it. Both
runs give the same tokens; the second takes fewer passes.
"""
from __future__ import annotations

import math
import os
import random
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import local_linear_attention_gb300 as lla  # noqa: E402


class Model:
    """Layers of attention with a residual; greedy tokens."""

    def __init__(self, layers=2, vocab=97, q_heads=4, kv_heads=2, d=32, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device=device) / math.sqrt(s[0])  # noqa: E731
        width = q_heads * d
        self.shape, self.h, self.spec = (q_heads, kv_heads, d), math.sqrt(d), lla.RotarySpec(d, base=1000.0)
        self.embed, self.head = rnd(vocab, width) * math.sqrt(vocab), rnd(width, vocab)
        self.layers = [{"q": rnd(width, width), "r": rnd(width, width) / d, "k": rnd(width, kv_heads * d),
                        "v": rnd(width, kv_heads * d), "out": rnd(width, width)} for _ in range(layers)]

    def next_tokens(self, tokens, caches, starts, max_new, parents=None, offsets=None):
        """The greedy token behind each of `tokens`, which go into the caches."""
        q_heads, kv_heads, d = self.shape
        x = self.embed[tokens]
        for w, cache in zip(self.layers, caches):
            y = x / x.norm(dim=-1, keepdim=True) * math.sqrt(x.shape[-1])
            q, k, v, r = ((y @ w[n]).view(len(tokens), -1, d) for n in "qkvr")
            q, r = lla.lla_paged_append_rotary(k, v, cache, starts, self.spec, q, r, offsets)
            if parents is None:
                out, _ = lla.lla_paged_attention(q, cache, starts, self.h, r=r, max_new=max_new)
            else:
                out, _ = lla.lla_paged_tree_attention(q, cache, starts, parents, self.h, r=r, max_new=max_new)
            x = x + out.view(len(tokens), -1) @ w["out"]
        return (x @ self.head).argmax(-1).tolist()


class Pages:
    """The pool of every layer, and how many table entries hold each page."""

    def __init__(self, model, num_pages, page, device="cuda"):
        _, kv_heads, d = model.shape
        self.pools = [[torch.zeros(num_pages, kv_heads, page, d, device=device) for _ in range(2)] for _ in model.layers]
        self.refs = torch.zeros(num_pages, dtype=torch.int32, device=device)

    def sequences(self, count, max_pages):
        """Caches of the layers for `count` empty sequences."""
        table = torch.zeros(count, max_pages, dtype=torch.int32, device=self.refs.device)
        lens = torch.zeros(count, dtype=torch.int32, device=self.refs.device)
        return [lla.PagedCache(k, v, table, lens) for k, v in self.pools]

    def grow(self, caches, news):
        """Room for news[b] more positions; returns starts."""
        starts = ints([sum(news[:b]) for b in range(len(news) + 1)])
        copies, left = lla.lla_paged_grow(caches[0], starts, self.refs)
        for cache in caches:
            lla.lla_paged_copy(cache, cache, copies)
        if int(left) < 0:
            raise RuntimeError(f"{-int(left)} pages or entries of the table too few")
        return starts


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def fork(model, pages, prompt, samples, max_pages):
    """Samples of one prompt: it is run once, its pages are shared, and each sample begins with a token of its own."""
    one, many = pages.sequences(1, max_pages), pages.sequences(samples, max_pages)
    starts = pages.grow(one, [len(prompt)])
    first = model.next_tokens(prompt, one, starts, len(prompt))[-1]
    lla.lla_paged_fork(one[0], many[0], ints([0] * samples), pages.refs)
    lla.lla_paged_free(one[0], pages.refs)
    return many, [(first + s) % model.embed.shape[0] for s in range(samples)]


def decode(model, pages, caches, last, count):
    """`count` tokens of each sequence behind last[b], one a pass."""
    out = [[] for _ in last]
    for _ in range(count):
        starts = pages.grow(caches, [1] * len(last))
        last = model.next_tokens(last, caches, starts, 1)
        for o, token in zip(out, last):
            o.append(token)
    return out


def draft(rng, last, future, vocab, depth=5, false_turns=2):
    """(tokens, parents) of a tree whose root is the last token: a stretch of the guess `future`, now and then
    wrong, and false turns off it."""
    tokens, parents, at = [last], [-1], 0
    for token in future[:depth]:
        for _ in range(false_turns):
            tokens.append(rng.randrange(vocab))
            parents.append(at)
        tokens.append(token if rng.random() < 0.8 else rng.randrange(vocab))
        parents.append(at)
        at = len(tokens) - 1
    return tokens, parents


def decode_drafted(model, pages, caches, last, count, guesses, seed=0):
    """The same with drafts; returns (tokens, passes)."""
    rng, vocab = random.Random(seed), model.embed.shape[0]
    out, passes = [[] for _ in last], 0
    while min(map(len, out)) < count:
        trees = [draft(rng, t, g[len(o):], vocab) for t, o, g in zip(last, out, guesses)]
        starts = pages.grow(caches, [len(t) for t, _ in trees])
        depths = []
        for _, parents in trees:
            d = []
            for p in parents:
                d.append(0 if p < 0 else d[p] + 1)
            depths += d
        after = model.next_tokens([t for tokens, _ in trees for t in tokens], caches, starts,
                                  max(len(t) for t, _ in trees), ints([p for _, parents in trees for p in parents]), ints(depths))
        paths, base = [], 0
        for b, (tokens, parents) in enumerate(trees):
            path, token = [0], after[base]
            while True:
                out[b].append(token)
                child = [i for i, p in enumerate(parents) if p == path[-1] and tokens[i] == token]
                if not child:
                    break
                path.append(child[0])
                token = after[base + child[0]]
            last[b] = token
            paths.append(path)
            base += len(tokens)
        longest = max(map(len, paths))
        path = ints([p + [-1] * (longest - len(p)) for p in paths])
        for cache in caches:
            keep = lla.lla_paged_compact(cache, starts, path)
        lla.lla_paged_free(caches[0], pages.refs, keep)
        passes += 1
    return out, passes


def serve(prompt_tokens=45, samples=3, count=40, page=16, seed=0):
    """Runs the example; returns (both runs' tokens, passes of the drafted one, pages held at the end)."""
    model = Model(seed=seed)
    pages = Pages(model, 64, page)
    rng = random.Random(seed)
    prompt = [rng.randrange(model.embed.shape[0]) for _ in range(prompt_tokens)]
    max_pages = -(-(prompt_tokens + count + 40) // page)
    plain, first = fork(model, pages, prompt, samples, max_pages)
    tokens = decode(model, pages, plain, list(first), count)
    drafted, first = fork(model, pages, prompt, samples, max_pages)
    again, passes = decode_drafted(model, pages, drafted, list(first), count, tokens, seed)
    lla.lla_paged_free(plain[0], pages.refs)
    lla.lla_paged_free(drafted[0], pages.refs)
    held = int((pages.refs != 0).sum())
    if lla.lla_stream_status() != 0:
        raise RuntimeError("liblla reported an error")
    return tokens, [o[:count] for o in again], passes, held


if __name__ == "__main__":
    tokens, again, passes, held = serve()
    print(f"{len(tokens[0])} tokens of {len(tokens)} samples in {passes} passes with drafts, the same: {tokens == again}; "
          f"pages held at the end: {held}")
