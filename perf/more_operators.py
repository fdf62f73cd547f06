"""The operators of drafting and branching on a paged cache, as cases to time and compare: attention of
a tree of drafted tokens (softmax or Parallax), rotary positions of queries, keys and probes with
their gradient, the append that rotates on the way, forking sequences that share pages until they
grow, and keeping one path of a drafted tree.

A case is a dict of plain values; `prepare` makes its inputs on the GPU, `run` does one pass (the
plain torch form, or the package's kernels where `own` is true) and `exact` gives the same outputs
from the definitions in float64.

Layouts: the cache is pages [num_pages, kv_heads, page_size, d]; sequence b's position j is slot
j % page_size of page page_table[b, j // page_size]; lens[b] counts its positions. New tokens of
all sequences lie one after the other, [tokens, heads, d], sequence b's at starts[b]..starts[b+1]-1,
and are the last positions of the sequence. refs[page] counts the table entries that hold a page.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- cases
def _case(op, **kw):
    base = {"op": op, "dtype": "bf16", "Hq": 8, "Hkv": 8, "d": 64, "dv": 64, "page": 64, "B": 1,
            "new_min": 1, "new_max": 1, "len_min": 1, "len_max": 1, "sizes": 0}
    extra = {"tree": {"window": 0, "sinks": 0, "probe": False, "branch": 2},
             "rotary": {"T": 1, "tensors": 3, "backward": False, "far": 0},
             "append": {"probe": False, "branch": 0, "far": 0},
             "branch": {"from": 1, "mass": False},
             "accept": {"path_max": 1, "mass": False}}[op]
    if op in ("rotary", "append"):
        extra.update({"rot": 64, "layout": "halves", "base": 10000.0, "stretch": "none", "factor": 1.0,
                      "context": 4096})
    return {**base, **extra, **kw}


def listed():
    return [
        # One user's draft on a short context, Parallax heads of 64: the call whose latency a chat feels.
        _case("tree", name="tree_one_n12_L1000", len_min=1000, len_max=1000, new_min=12, new_max=12, probe=True),
        # A batch of users with drafts of 32 nodes, grouped heads of 128, at the decode benchmark's lengths.
        _case("tree", name="tree_B16_n32_L16384", B=16, Hq=32, Hkv=8, d=128, dv=128, len_min=4096, len_max=16384,
              new_min=32, new_max=32),
        # A wide search below one long document.
        _case("tree", name="tree_one_n256_L32768", Hq=32, Hkv=8, d=128, dv=128, page=128, len_min=32768,
              len_max=32768, new_min=256, new_max=256, branch=4),
        # Full precision, unequal head sizes, ragged trees, a window and first tokens.
        _case("tree", name="tree_f32_window_B3", dtype="f32", B=3, Hq=6, Hkv=2, d=64, dv=32, page=16, new_min=1,
              new_max=29, len_min=40, len_max=2047, window=700, sinks=4, probe=True, branch=3),
        # q, k and the probe of a training step at the headline shape (B4 H8 T4096 d64).
        _case("rotary", name="rotary_B4_H8_T4096", B=4, T=4096),
        # The gradients of a stretched model that rotates part of a head, full precision, odd length.
        _case("rotary", name="rotary_gradient_f32_T2047", dtype="f32", B=2, T=2047, tensors=2, rot=48,
              layout="interleaved", stretch="wavelengths", factor=8.0, backward=True, far=500000),
        # The rotations and cache writes that go with a drafting step and with prompts.
        _case("append", name="append_rotary_draft_B16", B=16, Hq=32, Hkv=8, d=128, dv=128, rot=128, new_min=32,
              new_max=32, len_min=4096, len_max=16384, branch=2),
        _case("append", name="append_rotary_prompt_B4_T4096", B=4, d=128, dv=128, page=16, rot=128,
              layout="interleaved", new_min=4000, new_max=4096, len_min=4096, len_max=5001, probe=True,
              stretch="base", factor=4.0),
        # A beam search step: eight beams of which some survive twice and some die.
        _case("branch", name="branch_beams_8", B=8, **{"from": 8}, page=16, len_min=777, len_max=777, mass=True),
        # Sixteen samples each from four long prompts.
        _case("branch", name="branch_64_of_4_L16384", B=64, **{"from": 4}, d=128, dv=128, len_min=9000,
              len_max=16384, new_min=1, new_max=70),
        # The accepted path of one user's draft, and of a batch's.
        _case("accept", name="accept_one_n12", len_min=1000, len_max=1000, new_min=12, new_max=12, path_max=5),
        _case("accept", name="accept_B64_n64", B=64, d=128, dv=128, page=32, len_min=1000, len_max=5000, new_min=64,
              new_max=64, path_max=12, mass=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0.0), _cost(c))
    while True:
        op = rng.choice(["tree", "tree", "tree", "rotary", "append", "branch", "accept"])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        d = rng.choice([64, 128])
        c = _case(op, Hkv=Hkv, Hq=Hkv * rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16]), d=d, dv=d,
                  page=rng.choice([16, 32, 64, 128, 256]), sizes=rng.randrange(1 << 30))
        if rng.random() < 0.25:
            c["dtype"] = "f32"
        if rng.random() < 0.15:
            c["d"], c["dv"] = rng.choice([(64, 32), (32, 32), (16, 64), (32, 128)])
        c["B"] = _log_int(rng, 1, 64)
        c["len_max"] = _log_int(rng, 64, 32768)
        c["len_min"] = max(1, int(c["len_max"] * rng.uniform(0.1, 1.0)))
        c["new_max"] = _log_int(rng, 1, 256)
        c["new_min"] = rng.choice([1, max(1, c["new_max"] // 2), c["new_max"]])
        if op == "tree":
            c["branch"], c["probe"] = rng.choice([1, 2, 2, 3, 4, 8]), rng.random() < 0.4
            if rng.random() < 0.3:
                c["window"], c["sinks"] = _log_int(rng, 4, 4096), rng.choice([0, 1, 4, 16, 100])
        if op in ("rotary", "append"):
            c["rot"] = rng.choice([c["d"], c["d"], c["d"] // 2, c["d"] * 3 // 4, c["d"] // 4 + 2])
            c["layout"] = rng.choice(["halves", "interleaved"])
            c["base"] = rng.choice([10000.0, 10000.0, 500000.0, 1000000.0])
            c["stretch"] = rng.choice(["none", "none", "positions", "base", "wavelengths"])
            c["factor"] = 1.0 if c["stretch"] == "none" else rng.choice([2.0, 4.0, 8.0, 32.0])
            c["far"] = rng.choice([0, 0, 100000, 1 << 24])
        if op == "rotary":
            c["B"], c["T"] = _log_int(rng, 1, 16), _log_int(rng, 1, 8192)
            c["tensors"], c["backward"] = rng.choice([1, 2, 3]), rng.random() < 0.5
        if op == "append":
            c["branch"] = rng.choice([0, 2, 3])
            c["probe"] = rng.random() < 0.4
            if not c["branch"]:
                c["B"] = _log_int(rng, 1, 12)
                c["new_max"] = min(c["len_max"], _log_int(rng, 1, 4096))
                c["new_min"] = rng.choice([1, c["new_max"]])
        if op == "branch":
            c["from"], c["mass"] = _log_int(rng, 1, 64), rng.random() < 0.5
            c["len_max"] = min(c["len_max"], 16384)
            c["len_min"] = min(c["len_min"], c["len_max"])
        if op == "accept":
            c["path_max"], c["mass"] = _log_int(rng, 1, 16), rng.random() < 0.5
        if _cost(c) > most[op] or _pool(c) > 2 << 30:
            continue
        if op != "tree" or c["dtype"] != "f32" or _cost(c) <= most[op] / 16:
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


def _forest(case, news):
    """Each sequence's drafted tree: every node's parent (-1: the last token that is not drafted)."""
    rng = random.Random(case["sizes"] + 1)
    trees = []
    for t in news:
        parents = []
        for i in range(t):
            at = i // case["branch"] - 1
            parents.append(min(i - 1, max(-1, rng.randint(at - 1, at + 1))))
        trees.append(parents)
    return trees


def _depths(parents):
    depth = []
    for p in parents:
        depth.append(0 if p < 0 else depth[p] + 1)
    return depth


def _paths(case, trees):
    """A path of each tree, from a root to a node whose depth is near the case's longest."""
    rng = random.Random(case["sizes"] + 2)
    paths = []
    for parents in trees:
        depth = _depths(parents)
        most = rng.randint(0, min(case["path_max"], 1 + max(depth, default=-1)))
        path = []
        if most:
            at = rng.choice([i for i, x in enumerate(depth) if x == most - 1])
            while at >= 0:
                path.append(at)
                at = parents[at]
        paths.append(path[::-1])
    return paths


def _beams(case):
    """Lengths of the sequences forked from, and each new sequence's parent and number of new tokens."""
    rng = random.Random(case["sizes"] + 3)
    lens = [rng.randint(case["len_min"], case["len_max"]) for _ in range(case["from"])]
    parents = [rng.randrange(case["from"]) for _ in range(case["B"])]
    news = [rng.randint(case["new_min"], case["new_max"]) for _ in range(case["B"])]
    return lens, parents, news


def _pages(case, n):
    return (n + case["page"] - 1) // case["page"]


def _page_bytes(case):
    eb = 2 if case["dtype"] == "bf16" else 4
    return case["Hkv"] * case["page"] * ((case["d"] + case["dv"]) * eb + (4 if case.get("mass") else 0))


def _num_pages(case):
    if case["op"] == "branch":
        lens, parents, news = _beams(case)
        used = sum(_pages(case, n) for n in lens) + sum(
            _pages(case, lens[p] + t) - _pages(case, lens[p]) + 1 for p, t in zip(parents, news))
    else:
        used = sum(_pages(case, n) for n in _sizes(case)[0])
    return used + max(1, used // 16)


def _pool(case):
    return 0 if case["op"] == "rotary" else _num_pages(case) * _page_bytes(case)


def work(case):
    eb = 2 if case["dtype"] == "bf16" else 4
    Hq, Hkv, d, dv = case["Hq"], case["Hkv"], case["d"], case["dv"]
    if case["op"] == "rotary":
        n = case["tensors"] * case["B"] * Hq * case["T"] * d
        positions = 4 * case["B"] * case["T"] if case["far"] else 0
        return {"bytes": 2 * n * eb + positions, "flops": 3 * n}
    if case["op"] == "branch":
        lens, parents, news = _beams(case)
        copies = 0
        for p in range(case["from"]):
            children = parents.count(p)
            if lens[p] % case["page"]:
                copies += max(0, children - 1)
        entries = sum(_pages(case, n) for n in lens)
        for p, t in zip(parents, news):
            entries += _pages(case, lens[p] + t)
        return {"bytes": 4 * entries + 8 * _num_pages(case) + 2 * copies * _page_bytes(case), "flops": 0}
    lens, news = _sizes(case)
    tokens = sum(news)
    if case["op"] == "append":
        rows = Hkv * (d + dv) + Hq * d * (2 if case["probe"] else 1)
        return {"bytes": 2 * tokens * rows * eb + (4 * tokens if case["branch"] or case["far"] else 0),
                "flops": 3 * tokens * (Hkv + Hq * (2 if case["probe"] else 1)) * d}
    if case["op"] == "accept":
        moved = sum(a != i for path in _paths(case, _forest({**case, "branch": 3}, news)) for i, a in enumerate(path))
        return {"bytes": 2 * (tokens + moved) * Hkv * (d + dv) * eb + 4 * tokens, "flops": 0}
    pairs, keys = 0, 0
    for n, t, parents in zip(lens, news, _forest(case, news)):
        first, window, sinks = n - t, case["window"] or n + t, case["sinks"]
        for dep in _depths(parents):
            recent = min(first, max(0, window - 1 - dep))
            pairs += recent + min(sinks, first - recent) + min(dep + 1, window)
        recent = min(first, window - 1)
        keys += recent + min(sinks, first - recent) + t
    nbytes = tokens * (Hq * ((2 if case["probe"] else 1) * d * eb + dv * eb + 4) + 4) + keys * Hkv * (d + dv) * eb
    return {"bytes": nbytes, "flops": 2 * pairs * Hq * (d + dv) * (2 if case["probe"] else 1)}


def _cost(case):
    w = work(case)
    return w["bytes"] / 6e12 + w["flops"] / 1e15


# ------------------------------------------------------------------------------------ inputs
def _rand(gen, *shape, dtype=torch.bfloat16, scale=1.0):
    x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x * scale if scale != 1.0 else x).to(dtype)


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _frequencies(case):
    """The rotation per position of each pair, and the factor on what is rotated, from the formulas."""
    half, base, factor = case["rot"] // 2, case["base"], case["factor"]
    if case["stretch"] == "base":
        base *= factor ** (case["rot"] / (case["rot"] - 2))
    freq = [base ** (-2 * i / case["rot"]) for i in range(half)]
    scale = 1.0
    if case["stretch"] == "positions":
        freq = [f / factor for f in freq]
    elif case["stretch"] == "wavelengths":
        kept = [min(1.0, max(0.0, (case["context"] * f / (2 * math.pi) - 1) / 31)) for f in freq]
        freq = [f * (g + (1 - g) / factor) for f, g in zip(freq, kept)]
        scale = 0.1 * math.log(factor) + 1
    return freq, scale


def _spec(case):
    """The package's description of the same rotation."""
    import local_linear_attention_gb300 as lla
    return lla.RotarySpec(
        case["rot"], layout=lla.ROTARY_HALVES if case["layout"] == "halves" else lla.ROTARY_INTERLEAVED,
        base=case["base"], factor=case["factor"], context=case["context"], slow=1.0, fast=32.0,
        stretch={"none": lla.STRETCH_NONE, "positions": lla.STRETCH_POSITIONS, "base": lla.STRETCH_BASE,
                 "wavelengths": lla.STRETCH_WAVELENGTHS}[case["stretch"]])


def _table(order, counts, width=None):
    table = torch.zeros(len(counts), width or max(counts), dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    return table


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, page = _DTYPES[case["dtype"]], case["page"]
    Hq, Hkv, d, dv = case["Hq"], case["Hkv"], case["d"], case["dv"]
    s = {"case": case}
    if case["op"] in ("rotary", "append"):
        s["freq"], s["scale"] = _frequencies(case)
        s["spec"] = _spec(case) if own else None
    if case["op"] == "rotary":
        s["x"] = [_rand(gen, case["B"], Hq, case["T"], d, dtype=dtype) for _ in range(case["tensors"])]
        s["positions"] = None
        if case["far"]:  # packed documents and far continuations: each row's positions start somewhere
            start = torch.randint(0, case["far"], (case["B"], 1), generator=gen, device="cuda")
            s["positions"] = (start + torch.arange(case["T"], device="cuda")).to(torch.int32)
        return s
    # An allocator hands pages out in any order; one page in sixteen is free.
    num_pages = _num_pages(case)
    order = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    s["k_pages"] = _rand(gen, num_pages, Hkv, page, d, dtype=dtype)
    s["v_pages"] = _rand(gen, num_pages, Hkv, page, dv, dtype=dtype)
    s["mass"] = torch.rand(num_pages, Hkv, page, generator=gen, device="cuda") if case.get("mass") else None
    s["refs"] = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
    if case["op"] == "branch":
        lens, parents, news = _beams(case)
        s["lens_list"], s["parents_list"], s["news_list"] = lens, parents, news
        counts = [_pages(case, n) for n in lens]
        s["page_table"], s["lens"], s["parents"] = _table(order, counts), _int32(lens), _int32(parents)
        s["refs"][order[:sum(counts)].long()] = 1
        width = max(_pages(case, lens[p] + t) for p, t in zip(parents, news))
        s["to_table"] = torch.zeros(case["B"], max(width, max(counts)), dtype=torch.int32, device="cuda")
        s["to_lens"] = torch.zeros(case["B"], dtype=torch.int32, device="cuda")
        s["starts"] = _int32([sum(news[:b]) for b in range(case["B"] + 1)])
        return s
    lens, news = _sizes(case)
    counts = [_pages(case, n) for n in lens]
    s["page_table"], s["lens"] = _table(order, counts), _int32(lens)
    s["refs"][order[:sum(counts)].long()] = 1
    starts = [sum(news[:b]) for b in range(case["B"] + 1)]
    s.update({"lens_list": lens, "news_list": news, "starts_list": starts, "starts": _int32(starts),
              "max_new": max(news)})
    tokens = starts[-1]
    probe = case.get("probe")
    if case["op"] in ("tree", "append"):
        s["q"] = _rand(gen, tokens, Hq, d, dtype=dtype)
        s["r"] = _rand(gen, tokens, Hq, d, dtype=dtype, scale=1 / math.sqrt(d)) if probe else None
    if case["op"] in ("append", "accept"):
        s["k"] = _rand(gen, tokens, Hkv, d, dtype=dtype)
        s["v"] = _rand(gen, tokens, Hkv, dv, dtype=dtype)
    if case["op"] == "tree":
        s["h"] = math.sqrt(d)
        s["trees"] = _forest(case, news)
        s["parents"] = _int32([p for tree in s["trees"] for p in tree])
    if case["op"] == "append":
        s["offsets"] = None
        if case["branch"] or case["far"]:
            # drafted nodes sit at their depth, and eviction has dropped `far` positions at most
            gone = torch.randint(0, case["far"] + 1, (case["B"],), generator=gen, device="cuda").tolist()
            trees = _forest(case, news) if case["branch"] else None
            s["offsets"] = _int32([gone[b] + x for b, t in enumerate(news)
                                   for x in (_depths(trees[b]) if trees else range(t))])
    if case["op"] == "accept":
        s["paths"] = _paths(case, _forest({**case, "branch": 3}, news))
        s["path"] = _int32([p + [-1] * (case["path_max"] - len(p)) for p in s["paths"]])
    return s


# -------------------------------------------------------------------------------- plain forms
def _gathered(pages, row, n):
    """One sequence's positions of a paged array [pages, heads, page, ...], as [heads, n, ...]."""
    x = pages[row[:(n + pages.shape[2] - 1) // pages.shape[2]].long()].transpose(0, 1)
    return x.reshape(x.shape[0], -1, *x.shape[3:])[:, :n]


def _tree_mask(case, parents, n):
    """Which of n positions each node of a tree sees: [nodes, n]."""
    t, first = len(parents), n - len(parents)
    up = torch.tensor(parents, device="cuda")
    i = torch.arange(t, device="cuda")
    chain, depth, at = torch.zeros(t, t, dtype=torch.bool, device="cuda"), torch.zeros_like(i), i.clone()
    for _ in range(1 + max(_depths(parents))):
        alive = at >= 0
        chain[i[alive], at[alive]] = True
        at = torch.where(alive, up[at.clamp_min(0)], at)
        depth += (at >= 0).long()
    pos = first + depth
    seen = torch.cat([torch.ones(t, first, dtype=torch.bool, device="cuda"), chain], 1)
    if case["window"]:
        of_key = torch.cat([torch.arange(first, device="cuda"), pos])
        seen &= (of_key[None] > pos[:, None] - case["window"]) | (of_key[None] < case["sinks"])
    return seen


def _tree_plain(s):
    case = s["case"]
    Hq, Hkv, dv = case["Hq"], case["Hkv"], case["dv"]
    g = Hq // Hkv
    tokens = s["q"].shape[0]
    out = torch.zeros(tokens, Hq, dv, device="cuda")
    lse = torch.full((tokens, Hq), -math.inf, device="cuda")
    for b, (n, t) in enumerate(zip(s["lens_list"], s["news_list"])):
        at, row = s["starts_list"][b], s["page_table"][b]
        k = _gathered(s["k_pages"], row, n).float()[:, None]
        v = _gathered(s["v_pages"], row, n).float()[:, None]
        seen = _tree_mask(case, s["trees"][b], n)
        heads = lambda x: x[at:at + t].float().reshape(t, Hkv, g, -1).permute(1, 2, 0, 3)  # noqa: E731,B023
        logits = ((heads(s["q"]) @ k.transpose(-1, -2)) / s["h"]).masked_fill_(~seen, -math.inf)
        top = logits.amax(-1, keepdim=True)
        p = torch.exp(logits - top)
        total = p.sum(-1, keepdim=True)
        p = p / total
        lse[at:at + t] = (top + torch.log(total))[..., 0].permute(2, 0, 1).reshape(t, Hq)
        if case["probe"]:
            probe = heads(s["r"]) @ k.transpose(-1, -2)
            p = p * (1 + (p * probe).sum(-1, keepdim=True) - probe)
        out[at:at + t] = (p @ v).permute(2, 0, 1, 3).reshape(t, Hq, dv)
    return out.to(s["q"].dtype), lse


def _turned(s, x, angle):
    """x [..., d] with its first features rotated by `angle` [..., rot/2] (float64, as long positions need)."""
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    cos, sin = (torch.cos(angle) * s["scale"]).float(), (torch.sin(angle) * s["scale"]).float()
    if case.get("backward"):
        sin = -sin
    y = x.float().clone()
    first, second = (slice(0, half), slice(half, rot)) if case["layout"] == "halves" else \
        (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., first].float(), x[..., second].float()
    y[..., first], y[..., second] = a * cos - b * sin, a * sin + b * cos
    return y.to(x.dtype)


def _rotary_plain(s):
    case = s["case"]
    pos = torch.arange(case["T"], device="cuda")[None] if s["positions"] is None else s["positions"]
    angle = pos.double()[..., None] * torch.tensor(s["freq"], dtype=torch.float64, device="cuda")
    return [_turned(s, x, angle[:, None]) for x in s["x"]]


def _new_positions(s):
    """Each new token's sequence and slot's position."""
    news = s["starts"][1:] - s["starts"][:-1]
    tokens = s["starts_list"][-1]
    b = torch.repeat_interleave(torch.arange(s["case"]["B"], device="cuda"), news, output_size=tokens)
    return b, (s["lens"] - news)[b], torch.arange(tokens, device="cuda") - s["starts"][b]


def _write_plain(s, k):
    b, first, i = _new_positions(s)
    j, page = first + i, s["case"]["page"]
    at = s["page_table"][b, j // page].long()
    s["k_pages"][at, :, j % page] = k
    s["v_pages"][at, :, j % page] = s["v"]
    if s["mass"] is not None:
        s["mass"][at, :, j % page] = 0


def _append_plain(s):
    _, first, i = _new_positions(s)
    pos = first + (i if s["offsets"] is None else s["offsets"])
    angle = pos.double()[:, None, None] * torch.tensor(s["freq"], dtype=torch.float64, device="cuda")
    _write_plain(s, _turned(s, s["k"], angle))
    out = [s["k_pages"], s["v_pages"], _turned(s, s["q"], angle)]
    return out if s["r"] is None else out + [_turned(s, s["r"], angle)]


def _branch_plain(s):
    case, page = s["case"], s["case"]["page"]
    refs, table, old = s["refs"].clone(), s["to_table"], s["page_table"]
    one = torch.ones(old.shape[1], dtype=torch.int32, device="cuda")
    for c, p in enumerate(s["parents_list"]):
        m = _pages(case, s["lens_list"][p])
        table[c, :m] = old[p, :m]
        refs.index_add_(0, old[p, :m].long(), one[:m])
    for p, n in enumerate(s["lens_list"]):
        m = _pages(case, n)
        refs.index_add_(0, old[p, :m].long(), -one[:m])
    free = (refs == 0).nonzero()[:, 0].to(torch.int32)
    copies = torch.full((case["B"], 2), -1, dtype=torch.int32, device="cuda")
    used = 0
    for c, (p, t) in enumerate(zip(s["parents_list"], s["news_list"])):
        n = s["lens_list"][p]
        m = _pages(case, n)
        if t and n % page and int(refs[table[c, m - 1].long()]) > 1:
            copies[c, 0], copies[c, 1] = table[c, m - 1], free[used]
            refs[table[c, m - 1].long()] -= 1
            table[c, m - 1] = free[used]
            used += 1
        more = _pages(case, n + t) - m
        table[c, m:m + more] = free[used:used + more]
        used += more
        s["to_lens"][c] = n + t
    refs[free[:used].long()] = 1
    made = copies[copies[:, 0] >= 0].long()
    for x in (s["k_pages"], s["v_pages"], s["mass"]):
        if x is not None:
            x[made[:, 1]] = x[made[:, 0]]
    left = _int32([free.shape[0] - used])
    return [table, s["to_lens"], refs, copies, left] + _pools(s)


def _pools(s):
    return [x for x in (s["k_pages"], s["v_pages"], s["mass"]) if x is not None]


def _accept_plain(s):
    case, page = s["case"], s["case"]["page"]
    _write_plain(s, s["k"])
    refs, lens = s["refs"].clone(), s["lens"].clone()
    for b, path in enumerate(s["paths"]):
        n, first, row = s["lens_list"][b], s["lens_list"][b] - s["news_list"][b], s["page_table"][b].long()
        if path:
            src = first + torch.tensor(path, device="cuda")
            dst = first + torch.arange(len(path), device="cuda")
            for x in _pools(s):
                x[row[dst // page], :, dst % page] = x[row[src // page], :, src % page]
        refs[row[_pages(case, first + len(path)):_pages(case, n)]] -= 1
        lens[b] = first + len(path)
    return [lens.clone(), lens, refs] + _pools(s)


def run(state):
    case = state["case"]
    if not own:
        return {"tree": _tree_plain, "rotary": _rotary_plain, "append": _append_plain, "branch": _branch_plain,
                "accept": _accept_plain}[case["op"]](state)
    import local_linear_attention_gb300 as lla
    if case["op"] == "rotary":
        return lla.lla_rotary(state["x"], state["spec"], positions=state["positions"], backward=case["backward"])
    if case["op"] == "tree":
        cache = lla.PagedCache(state["k_pages"], state["v_pages"], state["page_table"], state["lens"])
        return lla.lla_paged_tree_attention(
            state["q"], cache, state["starts"], state["parents"], state["h"], r=state["r"], max_new=state["max_new"],
            window=case["window"], sinks=case["sinks"])
    if case["op"] == "append":
        cache = lla.PagedCache(state["k_pages"], state["v_pages"], state["page_table"], state["lens"])
        turned = lla.lla_paged_append_rotary(state["k"], state["v"], cache, state["starts"], state["spec"], state["q"],
                                             r=state["r"], offsets=state["offsets"])
        return [state["k_pages"], state["v_pages"], *(x for x in turned if x is not None)]
    refs, lens = state["refs"].clone(), state["lens"].clone()
    cache = lla.PagedCache(state["k_pages"], state["v_pages"], state["page_table"], lens, state["mass"])
    if case["op"] == "branch":
        to = lla.PagedCache(state["k_pages"], state["v_pages"], state["to_table"], state["to_lens"], state["mass"])
        lla.lla_paged_fork(cache, to, state["parents"], refs)
        lla.lla_paged_free(cache, refs)
        copies, left = lla.lla_paged_grow(to, state["starts"], refs)
        lla.lla_paged_copy(to, to, copies)
        return [state["to_table"], state["to_lens"], refs, copies, left] + _pools(state)
    lla.lla_paged_append(state["k"], state["v"], cache, state["starts"])
    keep = lla.lla_paged_compact(cache, state["starts"], state["path"])
    lla.lla_paged_free(cache, refs, keep)
    return [keep, lens, refs] + _pools(state)


# ------------------------------------------------------------------------------- the definition
def _exact_tree(case, s):
    page, Hkv, g = case["page"], case["Hkv"], case["Hq"] // case["Hkv"]
    tokens = s["q"].shape[0]
    out = torch.zeros(tokens, case["Hq"], case["dv"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(tokens, case["Hq"], dtype=torch.float64, device="cuda")
    for b, (n, t) in enumerate(zip(s["lens_list"], s["news_list"])):
        first, tree = n - t, s["trees"][b]
        blind = torch.zeros(t, n, dtype=torch.bool)
        level = [0] * t
        for i in range(t):
            level[i] = 0 if tree[i] < 0 else level[tree[i]] + 1
            line, a = {i}, tree[i]
            while a >= 0:
                line.add(a)
                a = tree[a]
            blind[i, first:] = torch.tensor([a not in line for a in range(t)])
        if case["window"]:
            at = torch.tensor(list(range(first)) + [first + x for x in level])
            mine = torch.tensor([first + x for x in level])[:, None]
            blind |= (mine - at >= case["window"]) & (at >= case["sinks"])
        blind = blind.cuda()
        j = torch.arange(n, device="cuda")
        src = s["page_table"][b].long()[j // page]
        rows = s["starts_list"][b] + torch.arange(t, device="cuda")
        for h in range(Hkv):
            k = s["k_pages"][src, h, j % page].double()
            v = s["v_pages"][src, h, j % page].double()
            for u in range(h * g, h * g + g):
                z = torch.mm(s["q"][rows, u].double(), k.T).div_(s["h"]).masked_fill_(blind, -math.inf)
                lse[rows, u] = torch.logsumexp(z, -1)
                w = torch.softmax(z, -1)
                o = w @ v
                if case["probe"]:
                    y = torch.mm(s["r"][rows, u].double(), k.T)
                    o = o - ((w * y) @ v - (w * y).sum(-1, keepdim=True) * o)
                out[rows, u] = o
    return out, lse


def _exact_turn(case, s, x, pos):
    """Pairs as complex numbers times scale * exp(i a), or its conjugate for the gradient."""
    freq = torch.tensor(s["freq"], dtype=torch.float64, device="cuda")
    unit = torch.polar(torch.full_like(freq, s["scale"]).expand(*pos.shape, -1).contiguous(),
                       pos.double()[..., None] * freq * (-1.0 if case.get("backward") else 1.0))
    rot = case["rot"]
    x = x.double()
    if case["layout"] == "halves":
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * unit
        return torch.cat([z.real, z.imag, x[..., rot:]], -1)
    z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2).contiguous()) * unit
    return torch.cat([torch.view_as_real(z).reshape(*x.shape[:-1], rot), x[..., rot:]], -1)


def _exact_branch(case, s):
    page = case["page"]
    table, count = s["page_table"].tolist(), s["refs"].tolist()
    lens, new_table = s["lens_list"], s["to_table"].tolist()
    held = [row[:-(-n // page)] for row, n in zip(table, lens)]
    rows = [list(held[p]) for p in s["parents_list"]]
    for row in rows:
        for x in row:
            count[x] += 1
    for row in held:
        for x in row:
            count[x] -= 1
    spare = [x for x, c in enumerate(count) if c == 0]
    copies = []
    for c, t in enumerate(s["news_list"]):
        n, row, pair = lens[s["parents_list"][c]], rows[c], [-1, -1]
        if t > 0 and n % page and count[row[-1]] > 1:
            count[row[-1]] -= 1
            pair = [row[-1], spare.pop(0)]
            row[-1] = pair[1]
            count[pair[1]] = 1
        while len(row) * page < n + t:
            row.append(spare.pop(0))
            count[row[-1]] = 1
        copies.append(pair)
        new_table[c][:len(row)] = row
    pools = [x.clone() for x in _pools(s)]
    for a, b in copies:
        if a >= 0:
            for x in pools:
                x[b] = x[a]
    grown = [lens[p] + t for p, t in zip(s["parents_list"], s["news_list"])]
    return [_int32(new_table), _int32(grown), _int32(count), _int32(copies), _int32([len(spare)])] + \
        [x.double() for x in pools]


def exact(case, seed):
    """The outputs of `run`, from the definitions in float64."""
    if case["op"] == "tree" and work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(case, s)
    if case["op"] == "rotary":
        pos = s["positions"]
        if pos is None:
            pos = torch.arange(case["T"], device="cuda").expand(case["B"], -1)
        return [_exact_turn(case, s, x, pos[:, None]) for x in s["x"]]
    if case["op"] == "branch":
        return _exact_branch(case, s)
    page, pools = case["page"], _pools(s)
    turned = case["op"] == "append"
    pools = [x.double() for x in pools]
    rows = {"k": s["k"].double(), "v": s["v"].double()}
    gone = s["offsets"].tolist() if turned and s["offsets"] is not None else None
    at = []
    for b, t in enumerate(s["news_list"]):
        first = s["lens_list"][b] - t
        at += [first + (i if gone is None else gone[s["starts_list"][b] + i]) for i in range(t)]
    if turned:
        at = torch.tensor(at, device="cuda")
        rows = {"k": _exact_turn(case, s, s["k"], at[:, None]), "v": rows["v"],
                "q": _exact_turn(case, s, s["q"], at[:, None])}
        if s["r"] is not None:
            rows["r"] = _exact_turn(case, s, s["r"], at[:, None])
    lens, refs = list(s["lens_list"]), s["refs"].clone()
    for b, t in enumerate(s["news_list"]):
        first, lo = s["lens_list"][b] - t, s["starts_list"][b]
        row = s["page_table"][b].long()
        j = first + torch.arange(t, device="cuda")
        for x, name in zip(pools, ("k", "v")):
            x[row[j // page], :, j % page] = rows[name][lo:lo + t]
        if len(pools) > 2:
            pools[2][row[j // page], :, j % page] = 0
        if turned:
            continue
        path = s["paths"][b]
        dst = first + torch.arange(len(path), device="cuda")
        for x, name in zip(pools, ("k", "v")):
            x[row[dst // page], :, dst % page] = rows[name][[lo + a for a in path]]
        lens[b] = first + len(path)
        for x in row[-(-lens[b] // page):-(-s["lens_list"][b] // page)].tolist():
            refs[x] -= 1
    if turned:
        return pools + [rows[x] for x in ("q", "r") if x in rows]
    return [_int32(lens), _int32(lens), refs] + pools
