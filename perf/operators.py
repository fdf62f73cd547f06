"""The paged-cache operators, as cases to time and compare: appending new tokens to a paged
key/value cache, attention of a chunk of new tokens over it (softmax or Parallax, with a sliding
window and first tokens that stay visible, and the attention weight that each cached position
receives), and eviction of the positions that received the least.

A case is a dict of plain values; `prepare` makes its inputs on the GPU, `run` does one pass (the
plain torch form, or the package's kernels where `own` is true) and `exact` gives the same outputs
from the definitions in float64.

Layouts: the cache is pages [num_pages, kv_heads, page_size, d]; sequence b's position j is slot
j % page_size of page page_table[b, j // page_size]; lens[b] counts its positions. New tokens of
all sequences lie one after the other, [tokens, heads, d], sequence b's at starts[b]..starts[b+1]-1,
and are the last positions of the sequence.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- cases
def _case(op, **kw):
    base = {"op": op, "dtype": "bf16", "Hq": 8, "Hkv": 8, "d": 64, "dv": 64, "page": 64,
            "B": 1, "new_min": 1, "new_max": 1, "len_min": 1, "len_max": 1, "sizes": 0,
            "window": 0, "sinks": 0, "probe": False, "weight": False}
    base.update(kw)
    return base


def listed():
    return [
        # One user's next token on a short context: the call whose latency a chat feels.
        _case("attend", name="attend_one_token_L1000", len_min=1000, len_max=1000, probe=True),
        # A full decode batch at the decode benchmark's batch and length, grouped heads of 128,
        # softmax attention with the weights that eviction needs.
        _case("attend", name="attend_decode_B32_L16384", B=32, Hq=32, Hkv=8, d=128, dv=128,
              len_min=4096, len_max=16384, weight=True),
        # The same traffic for Parallax heads of 64, one key/value head per query head.
        _case("attend", name="attend_decode_probe_B32_L16384", B=32, len_min=2048, len_max=16384,
              page=16, probe=True),
        # A long chat kept cheap by a window of 1024 keys and 4 first tokens.
        _case("attend", name="attend_decode_window_B48_L32768", B=48, Hq=28, Hkv=4, d=128, dv=128,
              page=32, len_min=500, len_max=32768, window=1024, sinks=4),
        # One long document: a chunk of its prompt against what is cached already.
        _case("attend", name="attend_chunk_2048_L32768", Hq=32, Hkv=8, d=128, dv=128,
              new_min=2048, new_max=2048, len_min=32768, len_max=32768, page=128),
        # Whole prompts of the headline's shape (B4 H8 T4096 d64), Parallax, with the weights.
        _case("attend", name="attend_prompt_probe_B4_T4096", B=4, new_min=4096, new_max=4096,
              len_min=4096, len_max=4096, probe=True, weight=True),
        # A serving step: many sequences that decode, some that bring the next ragged chunk of
        # their prompt, under a window.
        _case("attend", name="attend_mixed_B24_window", B=24, Hq=20, Hkv=4, d=128, dv=128,
              page=16, new_min=1, new_max=777, len_min=900, len_max=9000, window=2000, sinks=16,
              sizes=1),
        # Full precision, unequal head sizes, odd lengths.
        _case("attend", name="attend_f32_chunk_37", dtype="f32", B=3, Hq=6, Hkv=2, d=64, dv=32,
              page=16, new_min=1, new_max=37, len_min=40, len_max=2047, probe=True, weight=True),
        # The cache writes that go with a decode step and with a prompt.
        _case("append", name="append_decode_B32", B=32, d=128, dv=128, len_min=4096, len_max=16384),
        _case("append", name="append_prompt_B4_T4096", B=4, d=128, dv=128, page=16, new_min=4000,
              new_max=4096, len_min=4096, len_max=5001),
        # One sequence cut to a quarter, and a batch that has outgrown its memory.
        _case("evict", name="evict_one_L4000", page=16, len_min=4000, len_max=4000, budget=1000,
              sinks=4, recent=128),
        _case("evict", name="evict_B16_L32768", B=16, d=128, dv=128, len_min=9000, len_max=32768,
              budget=8192, sinks=16, recent=1024),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    most = {"attend": 0.0, "append": 0.0, "evict": 0.0}
    for c in listed():
        most[c["op"]] = max(most[c["op"]], _cost(c))
    while True:
        op = rng.choice(["attend", "attend", "attend", "append", "evict"])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16])
        d = rng.choice([64, 128])
        c = _case(op, Hkv=Hkv, Hq=Hkv * group, d=d, dv=d, page=rng.choice([16, 32, 64, 128, 256]),
                  sizes=rng.randrange(1 << 30))
        c["len_max"] = _log_int(rng, 64, 32768)
        c["len_min"] = max(1, int(c["len_max"] * rng.uniform(0.1, 1.0)))
        kind = rng.choice(["decode", "decode", "chunk", "prompt"])
        if kind == "decode":
            c["B"] = _log_int(rng, 1, 64)
            c["new_max"] = rng.choice([1, 1, 1, 2, 4])
        else:
            c["B"] = _log_int(rng, 1, 12)
            c["new_max"] = c["len_max"] if kind == "prompt" else _log_int(rng, 2, 2048)
            c["new_max"] = min(c["new_max"], 4096)
            c["new_min"] = rng.choice([1, max(1, c["new_max"] // 2), c["new_max"]])
        if op == "attend":
            if rng.random() < 0.3:
                c["window"], c["sinks"] = _log_int(rng, 16, 4096), rng.choice([0, 1, 4, 16, 100])
            c["probe"], c["weight"] = rng.random() < 0.4, rng.random() < 0.4
            if rng.random() < 0.2:
                c["dtype"] = "f32"
            if rng.random() < 0.15:
                c["d"], c["dv"] = rng.choice([(64, 32), (32, 32), (16, 64), (32, 128)])
        elif op == "evict":
            c["budget"] = max(1, int(c["len_max"] * rng.uniform(0.1, 1.1)))
            c["sinks"] = min(c["budget"], rng.choice([0, 1, 4, 16]))
            c["recent"] = int((c["budget"] - c["sinks"]) * rng.choice([0.0, 0.1, 0.5]))
        if _cost(c) <= most[op] and _pool(c) <= 3 << 30 and (c["dtype"] != "f32" or _cost(c) <= most[op] / 16):
            return c


def _sizes(case):
    """Each sequence's length (its new tokens included) and number of new tokens."""
    rng = random.Random(case["sizes"])
    lens, news = [], []
    for b in range(case["B"]):
        n = rng.randint(case["len_min"], case["len_max"])
        if case["new_min"] < case["new_max"] and rng.random() < 0.6:
            t = case["new_min"]
        else:
            t = rng.randint(case["new_min"], case["new_max"])
        lens.append(n)
        news.append(min(t, n))
    return lens, news


def _pages(case, n):
    return (n + case["page"] - 1) // case["page"]


def _pool(case):
    lens, _ = _sizes(case)
    return sum(_pages(case, n) for n in lens) * case["page"] * case["Hkv"] * (case["d"] + case["dv"]) * 4


def _visible(case, n, t):
    """(pairs of a new token and a key it sees, keys that any new token sees) of one sequence."""
    window, sinks = case["window"] or n, case["sinks"]
    pairs = 0
    for i in range(n - t, n):
        recent = min(window, i + 1)
        pairs += recent + min(sinks, i + 1 - recent)
    first = max(0, n - t - window + 1)
    return pairs, n - first + min(sinks, first)


def work(case):
    eb = 2 if case["dtype"] == "bf16" else 4
    lens, news = _sizes(case)
    Hq, Hkv, d, dv = case["Hq"], case["Hkv"], case["d"], case["dv"]
    tokens = sum(news)
    if case["op"] == "append":
        return {"bytes": 2 * tokens * Hkv * (d + dv) * eb, "flops": 0}
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": Hkv * (4 * sum(lens) + kept * (2 * (d + dv) * eb + 8)), "flops": 0}
    seen = [_visible(case, n, t) for n, t in zip(lens, news)]
    pairs, keys = sum(s[0] for s in seen), sum(s[1] for s in seen)
    width = (d + dv) * (2 if case["probe"] else 1)
    nbytes = tokens * Hq * ((2 if case["probe"] else 1) * d * eb + dv * eb + 4)
    nbytes += keys * Hkv * ((d + dv) * eb + (8 if case["weight"] else 0))
    return {"bytes": nbytes, "flops": 2 * pairs * Hq * width}


def _cost(case):
    w = work(case)
    return w["bytes"] / 6e12 + w["flops"] / 1e14


# ------------------------------------------------------------------------------------ inputs
def _rand(gen, *shape, dtype=torch.bfloat16, scale=1.0):
    x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x * scale if scale != 1.0 else x).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens, news = _sizes(case)
    dtype, page = _DTYPES[case["dtype"]], case["page"]
    Hq, Hkv, d, dv = case["Hq"], case["Hkv"], case["d"], case["dv"]
    counts = [_pages(case, n) for n in lens]
    # An allocator hands pages out in any order; one page in sixteen is free.
    num_pages = sum(counts) + max(1, sum(counts) // 16)
    order = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(case["B"], max(counts), dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    starts = [0]
    for t in news:
        starts.append(starts[-1] + t)
    s = {"case": case, "lens_list": lens, "news_list": news, "starts_list": starts,
         "page_table": table, "max_new": max(news),
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "starts": torch.tensor(starts, dtype=torch.int32, device="cuda"),
         "k_pages": _rand(gen, num_pages, Hkv, page, d, dtype=dtype),
         "v_pages": _rand(gen, num_pages, Hkv, page, dv, dtype=dtype)}
    if case["op"] == "append":
        s["k"] = _rand(gen, starts[-1], Hkv, d, dtype=dtype)
        s["v"] = _rand(gen, starts[-1], Hkv, dv, dtype=dtype)
    if case["op"] == "attend":
        s["h"] = math.sqrt(d)
        s["q"] = _rand(gen, starts[-1], Hq, d, dtype=dtype)
        s["r"] = _rand(gen, starts[-1], Hq, d, dtype=dtype, scale=1 / math.sqrt(d)) if case["probe"] else None
        if case["weight"]:
            s["mass"] = torch.rand(num_pages, Hkv, page, generator=gen, device="cuda")
    if case["op"] == "evict":
        # Accumulated weights: a few positions hold most, and those that no row ever saw are zero.
        mass = torch.randn(num_pages, Hkv, page, generator=gen, device="cuda").mul_(2).exp_()
        s["mass"] = mass * (torch.rand(mass.shape, generator=gen, device="cuda") > 0.05)
        kept = [_pages(case, min(n, case["budget"])) for n in lens]
        order = torch.randperm(sum(kept), generator=gen, device="cuda").to(torch.int32)
        to = torch.zeros(case["B"], max(kept), dtype=torch.int32, device="cuda")
        at = 0
        for b, c in enumerate(kept):
            to[b, :c] = order[at:at + c]
            at += c
        s["to"] = {"page_table": to, "lens": torch.zeros(case["B"], dtype=torch.int32, device="cuda"),
                   "k_pages": torch.zeros(sum(kept), Hkv, page, d, dtype=dtype, device="cuda"),
                   "v_pages": torch.zeros(sum(kept), Hkv, page, dv, dtype=dtype, device="cuda"),
                   "mass": torch.zeros(sum(kept), Hkv, page, device="cuda")}
    return s


# -------------------------------------------------------------------------------- plain forms
def _gathered(pages, row, n):
    """One sequence's positions of a paged array [pages, heads, page, ...], as [heads, n, ...]."""
    x = pages[row[:(n + pages.shape[2] - 1) // pages.shape[2]].long()].transpose(0, 1)
    return x.reshape(x.shape[0], -1, *x.shape[3:])[:, :n]


def _mask(case, first, count, n):
    """Which of n positions the new tokens at positions first..first+count-1 see."""
    i = torch.arange(first, first + count, device="cuda")[:, None]
    j = torch.arange(n, device="cuda")[None, :]
    seen = j <= i
    if case["window"]:
        seen &= (j > i - case["window"]) | (j < case["sinks"])
    return seen


def _attend_plain(s):
    case = s["case"]
    Hq, Hkv, dv = case["Hq"], case["Hkv"], case["dv"]
    g = Hq // Hkv
    tokens = s["q"].shape[0]
    out = torch.zeros(tokens, Hq, dv, device="cuda")
    lse = torch.full((tokens, Hq), -math.inf, device="cuda")
    mass = s["mass"].clone() if case["weight"] else None
    for b, (n, t) in enumerate(zip(s["lens_list"], s["news_list"])):
        at, row = s["starts_list"][b], s["page_table"][b]
        k = _gathered(s["k_pages"], row, n).float()[:, None]
        v = _gathered(s["v_pages"], row, n).float()[:, None]
        received = torch.zeros(Hkv, n, device="cuda")
        step = max(1, (1 << 28) // (Hq * n))
        for a in range(0, t, step):
            e = min(t, a + step)
            heads = lambda x: x[at + a:at + e].float().reshape(e - a, Hkv, g, -1).permute(1, 2, 0, 3)
            logits = (heads(s["q"]) @ k.transpose(-1, -2)) / s["h"]
            logits.masked_fill_(~_mask(case, n - t + a, e - a, n), -math.inf)
            top = logits.amax(-1, keepdim=True)
            p = torch.exp(logits - top)
            total = p.sum(-1, keepdim=True)
            p = p / total
            lse[at + a:at + e] = (top + torch.log(total))[..., 0].permute(2, 0, 1).reshape(e - a, Hq)
            received += p.sum((1, 2))
            if case["probe"]:
                probe = heads(s["r"]) @ k.transpose(-1, -2)
                p = p * (1 + (p * probe).sum(-1, keepdim=True) - probe)
            out[at + a:at + e] = (p @ v).permute(2, 0, 1, 3).reshape(e - a, Hq, dv)
        if mass is not None:
            j = torch.arange(n, device="cuda")
            mass[row[j // case["page"]].long(), :, j % case["page"]] += received.T
    out = out.to(s["q"].dtype)
    return (out, lse) if mass is None else (out, lse, mass)


def _append_plain(s):
    case = s["case"]
    n = torch.repeat_interleave(s["lens"] - (s["starts"][1:] - s["starts"][:-1]),
                                s["starts"][1:] - s["starts"][:-1], output_size=s["k"].shape[0])
    b = torch.repeat_interleave(torch.arange(case["B"], device="cuda"),
                                s["starts"][1:] - s["starts"][:-1], output_size=s["k"].shape[0])
    j = n + torch.arange(s["k"].shape[0], device="cuda") - s["starts"][b]
    page = s["page_table"][b, j // case["page"]].long()
    s["k_pages"][page, :, j % case["page"]] = s["k"]
    s["v_pages"][page, :, j % case["page"]] = s["v"]
    return s["k_pages"], s["v_pages"]


def _evict_plain(s):
    case, to = s["case"], s["to"]
    Hkv, budget = case["Hkv"], case["budget"]
    kept = torch.full((case["B"], Hkv, budget), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(s["lens_list"]):
        m = min(n, budget)
        mass = _gathered(s["mass"], s["page_table"][b], n)
        rank = mass.clone()
        rank[:, :case["sinks"]] = math.inf
        rank[:, n - min(n, case["recent"]):] = math.inf
        best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[:, :m]
        best = torch.sort(best, dim=-1).values
        kept[b, :, :m] = best
        i = torch.arange(m, device="cuda")
        h = torch.arange(Hkv, device="cuda")[:, None]
        src = s["page_table"][b][best // case["page"]].long()
        dst = to["page_table"][b][i // case["page"]].long()[None, :]
        for name in ("k_pages", "v_pages", "mass"):
            to[name][dst, h, (i % case["page"])[None, :]] = s[name][src, h, best % case["page"]]
        to["lens"][b] = m
    return to["k_pages"], to["v_pages"], to["mass"], to["lens"], kept


def run(state):
    case = state["case"]
    if not own:
        return {"attend": _attend_plain, "append": _append_plain, "evict": _evict_plain}[case["op"]](state)
    import local_linear_attention_gb300 as lla
    if case["op"] == "append":
        cache = lla.PagedCache(state["k_pages"], state["v_pages"], state["page_table"], state["lens"])
        lla.lla_paged_append(state["k"], state["v"], cache, state["starts"])
        return state["k_pages"], state["v_pages"]
    if case["op"] == "attend":
        mass = state["mass"].clone() if case["weight"] else None
        cache = lla.PagedCache(state["k_pages"], state["v_pages"], state["page_table"], state["lens"], mass)
        out, lse = lla.lla_paged_attention(
            state["q"], cache, state["starts"], state["h"], r=state["r"], max_new=state["max_new"],
            window=case["window"], sinks=case["sinks"], track_mass=case["weight"])
        return (out, lse) if mass is None else (out, lse, mass)
    cache = lla.PagedCache(state["k_pages"], state["v_pages"], state["page_table"], state["lens"], state["mass"])
    to = state["to"]
    dest = lla.PagedCache(to["k_pages"], to["v_pages"], to["page_table"], to["lens"], to["mass"])
    kept = lla.lla_paged_evict(cache, dest, case["budget"], sinks=case["sinks"], recent=case["recent"])
    return to["k_pages"], to["v_pages"], to["mass"], to["lens"], kept


# ------------------------------------------------------------------------------- the definition
def exact(case, seed):
    """The outputs of `run`, from the definitions in float64: softmax weights over the visible
    positions and, with a probe r, mean(v) - Cov(v, k) r under those weights."""
    if case["op"] == "attend" and work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    page, Hkv = case["page"], case["Hkv"]
    if case["op"] == "append":
        for b in range(case["B"]):
            at, t = s["starts_list"][b], s["news_list"][b]
            for i in range(t):
                j = s["lens_list"][b] - t + i
                if i and j % page:
                    continue
                m = min(page - j % page, t - i)
                dst = int(s["page_table"][b, j // page])
                s["k_pages"][dst, :, j % page:j % page + m] = s["k"][at + i:at + i + m].transpose(0, 1)
                s["v_pages"][dst, :, j % page:j % page + m] = s["v"][at + i:at + i + m].transpose(0, 1)
        return s["k_pages"].double(), s["v_pages"].double()
    if case["op"] == "evict":
        kept = torch.full((case["B"], Hkv, case["budget"]), -1, dtype=torch.int32)
        to = s["to"]
        for b, n in enumerate(s["lens_list"]):
            m = min(n, case["budget"])
            tail = max(0, n - case["recent"])
            j = torch.arange(n, device="cuda")
            src, dst = s["page_table"][b].long(), to["page_table"][b].long()
            for h in range(Hkv):
                mass = s["mass"][src[j // page], h, j % page].tolist()
                order = sorted(range(n), key=lambda i: (0 if i < case["sinks"] or i >= tail else 1,
                                                        -mass[i] if case["sinks"] <= i < tail else 0.0, i))
                pick = torch.tensor(sorted(order[:m]), device="cuda")
                kept[b, h, :m] = pick.int().cpu()
                i = torch.arange(m, device="cuda")
                for name in ("k_pages", "v_pages", "mass"):
                    to[name][dst[i // page], h, i % page] = s[name][src[pick // page], h, pick % page]
            to["lens"][b] = m
        return to["k_pages"].double(), to["v_pages"].double(), to["mass"].double(), to["lens"], kept
    g = case["Hq"] // Hkv
    tokens = s["q"].shape[0]
    out = torch.zeros(tokens, case["Hq"], case["dv"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(tokens, case["Hq"], dtype=torch.float64, device="cuda")
    mass = s["mass"].double() if case["weight"] else None
    for b, (n, t) in enumerate(zip(s["lens_list"], s["news_list"])):
        j = torch.arange(n, device="cuda")
        src = s["page_table"][b].long()[j // page]
        for h in range(Hkv):
            k = s["k_pages"][src, h, j % page].double()
            v = s["v_pages"][src, h, j % page].double()
            got = torch.zeros(n, dtype=torch.float64, device="cuda")
            step = max(1, (1 << 25) // n)
            for a in range(0, t, step):
                i = torch.arange(a, min(t, a + step), device="cuda")
                pos, rows = (n - t + i)[:, None], s["starts_list"][b] + i
                blind = j[None, :] > pos
                if case["window"]:
                    blind = blind | ((pos - j[None, :] >= case["window"]) & (j[None, :] >= case["sinks"]))
                for u in range(g):
                    x = s["q"][rows, h * g + u].double()
                    z = torch.mm(x, k.T).div_(s["h"]).masked_fill_(blind, -math.inf)
                    lse[rows, h * g + u] = torch.logsumexp(z, -1)
                    w = torch.softmax(z, -1)
                    got += w.sum(0)
                    o = w @ v
                    if case["probe"]:
                        y = torch.mm(s["r"][rows, h * g + u].double(), k.T)
                        o = o - ((w * y) @ v - (w * y).sum(-1, keepdim=True) * o)
                    out[rows, h * g + u] = o
            if mass is not None:
                mass[src, h, j % page] += got
    return (out, lse) if mass is None else (out, lse, mass)
