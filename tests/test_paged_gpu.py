"""GPU tests of the paged-cache operators against the float64 reference (paged_reference.py), at the
sizes, masks and orders where they can go wrong. Tolerances are the reference's derived bounds."""
import math

import pytest
import torch

from paged_reference import Problem, attention, evict

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lla():
    from local_linear_attention_gb300 import binding, build
    build.build()
    return binding


def check(name, got, ref, tol):
    got, ref, tol = got.double().cpu(), ref.double(), tol.double()
    same = (got == ref) | (got.isnan() & ref.isnan())
    bad = ~same & ~((got - ref).abs() <= tol)
    if bad.any():
        i = tuple(int(x[0]) for x in bad.nonzero(as_tuple=True))
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} beyond tolerance, first at {i}: "
                             f"{float(got[i]):.9g} against {float(ref[i]):.9g}, tolerance {float(tol[i]):.3g}")


def run_and_check(lla, P, window=0, sinks=0, track=True, path=0, max_new=None, workspace=False):
    cache, q, r, starts = P.cuda(lla)
    ref = attention(P, window, sinks)
    kw = dict(r=r, max_new=max(P.news_l) if max_new is None else max_new, window=window, sinks=sinks,
              track_mass=track, path=path)
    if workspace:
        n = lla.lla_paged_workspace_size(q, cache, starts, P.h, **kw)
        kw["workspace"] = torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda")
    out, lse = lla.lla_paged_attention(q, cache, starts, P.h, **kw)
    assert lla.lla_stream_status() == 0
    check("out", out, ref["out"], ref["out_tol"])
    check("lse", lse, ref["lse"], ref["lse_tol"])
    if track:
        check("mass", cache.mass, ref["mass"], ref["mass_tol"])
    else:
        assert torch.equal(cache.mass.cpu(), P.mass)
    return out, lse, cache


# Ragged batches: single tokens, chunks, whole prompts, lengths of one, sequences without new
# tokens and without anything.
BATCHES = {
    "one": ([1], [1]),
    "decode": ([1, 17, 100, 533, 64], [1, 1, 1, 1, 1]),
    "few": ([5, 300, 129, 16], [4, 2, 3, 1]),
    "chunk": ([200, 77, 0, 700, 33], [65, 1, 0, 130, 33]),
    "idle": ([50, 60, 300], [0, 60, 0]),
}


@pytest.mark.parametrize("probe", [False, True])
@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("dtype,d,dv,Hq,Hkv,page", [
    (F32, 64, 64, 4, 2, 16), (F32, 16, 128, 3, 1, 64), (BF, 64, 64, 4, 4, 16), (BF, 128, 128, 8, 2, 32),
    (BF, 64, 64, 5, 1, 128), (BF, 128, 128, 21, 3, 256), (BF, 32, 16, 2, 1, 16), (BF, 128, 64, 6, 2, 64),
    (BF, 64, 64, 40, 2, 64), (BF, 16, 128, 4, 4, 16), (BF, 64, 32, 12, 4, 32), (BF, 16, 64, 30, 2, 128),
    (F32, 32, 16, 300, 2, 16), (BF, 64, 16, 260, 2, 16)])
def test_attention(lla, dtype, d, dv, Hq, Hkv, page, batch, probe):
    lens, news = BATCHES[batch]
    run_and_check(lla, Problem(lens, news, Hq, Hkv, d, dv, page, dtype, probe, seed=d + Hq + page))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (100, 0), (64, 130), (300, 5), (10000, 2)])
@pytest.mark.parametrize("batch", ["decode", "few", "chunk"])
@pytest.mark.parametrize("dtype,d,probe", [(F32, 32, True), (BF, 64, True), (BF, 128, False), (BF, 128, True),
                                           (BF, 64, False)])
def test_window_and_sinks(lla, dtype, d, probe, batch, window, sinks):
    lens, news = BATCHES[batch]
    run_and_check(lla, Problem(lens, news, 6, 2, d, d, 32, dtype, probe, seed=window + sinks), window, sinks)


@pytest.mark.parametrize("dtype,d,dv", [(BF, 64, 64), (BF, 128, 128), (F32, 64, 32), (BF, 16, 16)])
@pytest.mark.parametrize("probe", [False, True])
def test_long_sequences_split_over_blocks(lla, dtype, d, dv, probe):
    run_and_check(lla, Problem([9001, 4096, 3], [1, 1, 1], 4, 2, d, dv, 64, dtype, probe, seed=5), workspace=True)
    run_and_check(lla, Problem([5000], [70], 4, 2, d, dv, 16, dtype, probe, seed=6), track=True)
    run_and_check(lla, Problem([3333], [9], 2, 1, d, dv, 16, dtype, probe, seed=7), window=2500, sinks=50)


@pytest.mark.parametrize("dtype,d", [(F32, 64), (BF, 64), (BF, 128)])
def test_cuda_core_path(lla, dtype, d):
    for batch in ("decode", "chunk"):
        lens, news = BATCHES[batch]
        run_and_check(lla, Problem(lens, news, 6, 2, d, d, 16, dtype, True, seed=11), path=1, window=50, sinks=4)


@pytest.mark.parametrize("dtype,d,page", [(BF, 64, 16), (BF, 128, 64), (F32, 64, 16), (BF, 128, 1024)])
@pytest.mark.parametrize("lens,news", [([40, 100, 1], [1, 1, 1]), ([40, 300, 5], [3, 150, 5])])
@pytest.mark.parametrize("probe", [False, True])
def test_slots_nobody_sees_may_hold_anything(lla, dtype, d, page, lens, news, probe):
    """Free pages, the rest of a last page, and positions that fell out of the window."""
    P = Problem(lens, news, 4, 2, d, d, page, dtype, probe, seed=3)
    window, sinks = 20, 2
    junk = torch.tensor([math.nan, math.inf, -math.inf, torch.finfo(dtype).max, torch.finfo(dtype).min])
    used = torch.zeros(P.num_pages, page, dtype=torch.bool)
    for b, (n, t) in enumerate(zip(lens, news)):
        pg, off = P.slots(b)
        j = torch.arange(n)
        keep = (j < sinks) | (j > n - t - window)
        used[pg[keep], off[keep]] = True
    for x in (P.k, P.v):
        fill = junk[torch.arange(x.shape[-1]) % 5].to(dtype)
        x.copy_(torch.where(used[:, None, :, None], x, fill))
    run_and_check(lla, P, window, sinks)


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 32)])
@pytest.mark.parametrize("lens,news", [([70], [4]), ([400], [300])])
@pytest.mark.parametrize("probe", [False, True])
def test_a_value_that_is_not_finite_reaches_only_the_rows_that_see_it(lla, dtype, d, lens, news, probe):
    """The new tokens' keys and values: an infinite value at the last position and a NaN key in the
    middle of the chunk leave the earlier rows as they were."""
    P = Problem(lens, news, 2, 1, d, d, 16, dtype, probe, seed=8)
    n, t = lens[0], news[0]
    pg, off = P.slots(0)
    cut = n - t + t // 2
    P.v[pg[n - 1], 0, off[n - 1], 1] = math.inf
    P.k[pg[cut], 0, off[cut], 0] = math.nan
    clean = Problem(lens, news, 2, 1, d, d, 16, dtype, probe, seed=8)
    ref = attention(clean)
    cache, q, r, starts = P.cuda(lla)
    out, lse = lla.lla_paged_attention(q, cache, starts, P.h, r=r, max_new=t, track_mass=True)
    assert lla.lla_stream_status() == 0
    good = t // 2
    check("out", out[:good], ref["out"][:good], ref["out_tol"][:good])
    check("lse", lse[:good], ref["lse"][:good], ref["lse_tol"][:good])
    assert out[good:].isnan().all() and lse[good:].isnan().all()


@pytest.mark.parametrize("dtype,d,news", [(BF, 64, [300]), (BF, 128, [300]), (BF, 128, [1]), (F32, 32, [20])])
def test_a_key_that_is_not_finite_far_back(lla, dtype, d, news):
    """Every row sees it: all are NaN, and the call does not take its time over them."""
    P = Problem([30000], news, 8, 2, d, d, 64, dtype, False, seed=22)
    pg, off = P.slots(0)
    P.k[pg[7], 0, off[7], 0] = math.nan
    cache, q, r, starts = P.cuda(lla)
    begin, end = torch.cuda.Event(True), torch.cuda.Event(True)
    for _ in range(2):
        begin.record()
        out, lse = lla.lla_paged_attention(q, cache, starts, P.h, max_new=news[0])
        end.record()
    assert lla.lla_stream_status() == 0
    assert out[:, :4].isnan().all() and lse[:, :4].isnan().all()
    assert out[:, 4:].isfinite().all() and lse[:, 4:].isfinite().all()
    assert begin.elapsed_time(end) < 100.0  # ms; rows taken again one by one would need seconds


@pytest.mark.parametrize("probe", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_logits_that_grow_from_tile_to_tile(lla, d, probe):
    """Later keys outweigh everything before them by far more than the range of fp32."""
    P = Problem([1500], [260], 4, 2, d, d, 64, BF, probe, seed=23)
    pg, off = P.slots(0)
    scale = torch.linspace(0.1, 30.0, 1500) ** 2
    base = P.k[pg[0], 0, off[0]].clone()
    P.k[pg, 0, off] = (base[None] * scale[:, None]).bfloat16()
    P.q = (base.sign()[None, None] * P.q.abs()).bfloat16()  # q.k > 0 and growing with the position
    run_and_check(lla, P)


def test_more_sequences_than_the_tensor_core_kernel_schedules(lla):
    P = Problem([20 + i % 13 for i in range(2100)], [2] * 2100, 9, 1, 64, 64, 16, BF, False, seed=24)
    run_and_check(lla, P, track=False)


def test_workspace_of_a_chunk(lla):
    for d, probe in ((64, True), (128, False)):
        run_and_check(lla, Problem([900, 5000], [150, 300], 4, 2, d, d, 32, BF, probe, seed=25), workspace=True)


def test_rows_before_the_first_position_see_nothing(lla):
    """More new tokens than positions: the first rows have positions below zero."""
    for dtype, d, news in ((BF, 64, [5, 1]), (BF, 128, [200, 3]), (F32, 64, [70, 2])):
        P = Problem([3, 10], news, 2, 1, d, d, 16, dtype, True, seed=9)
        run_and_check(lla, P)
        cache, q, r, starts = P.cuda(lla)
        out, lse = lla.lla_paged_attention(q, cache, starts, P.h, r=r, max_new=max(news))
        empty = news[0] - 3
        assert (out[:empty] == 0).all() and (lse[:empty] == -math.inf).all()


def test_large_logits_and_equal_keys(lla):
    """Logits of thousands (one key takes all the weight) and none at all (uniform weights)."""
    for dtype, d in ((BF, 128), (BF, 64), (F32, 64)):
        for scale in (200.0, 0.0):
            for lens, news in (([130, 300], [1, 1]), ([130, 300], [40, 200])):
                P = Problem(lens, news, 4, 2, d, d, 32, dtype, True, seed=10)
                P.q = (P.q.float() * scale).to(dtype)
                run_and_check(lla, P)


def test_results_do_not_depend_on_the_run(lla):
    for dtype, d, news in ((BF, 64, [1, 1]), (BF, 128, [150, 1]), (F32, 64, [33, 1])):
        P = Problem([3000, 700], news, 8, 2, d, d, 64, dtype, True, seed=12)
        first = None
        for _ in range(3):
            out, lse, cache = run_and_check(lla, P)
            now = (out, lse, cache.mass)
            assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
            first = now


def test_matches_the_contiguous_operators(lla):
    """Whole prompts against lla_parallax_forward, single tokens against lla_parallax_decode."""
    T, H, d = 300, 3, 64
    P = Problem([T, T], [T, T], H, H, d, d, 16, BF, True, seed=13)
    cache, q, r, starts = P.cuda(lla)
    out, _ = lla.lla_paged_attention(q, cache, starts, P.h, r=r, max_new=T)
    k = torch.stack([P.k[P.slots(b)[0], :, P.slots(b)[1]] for b in range(2)]).transpose(1, 2).contiguous().cuda()
    v = torch.stack([P.v[P.slots(b)[0], :, P.slots(b)[1]] for b in range(2)]).transpose(1, 2).contiguous().cuda()
    heads = lambda x: x.reshape(2, T, H, d).transpose(1, 2).contiguous()  # noqa: E731
    full = lla.lla_parallax_forward(heads(q), k, v, heads(r), P.h)
    ref = attention(P)
    tol = ref["out_tol"].reshape(2, T, H, d).transpose(1, 2)
    check("forward", heads(out), full.cpu(), 2 * tol)
    last = torch.tensor([T - 1, 2 * T - 1], device="cuda")
    step = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    one, _ = lla.lla_paged_attention(q[last], cache, step, P.h, r=r[last], max_new=1)
    dec = lla.lla_parallax_decode(q[last], k, v, r[last], P.h)
    check("decode", one, dec.cpu(), 2 * tol[:, :, -1])


def test_append(lla):
    for dtype, d, dv, Hkv in ((BF, 64, 64, 3), (F32, 128, 16, 1), (BF, 16, 128, 2), (F32, 32, 64, 5)):
        P = Problem([70, 5, 33, 0, 3], [1, 5, 20, 0, 7], Hkv, Hkv, d, dv, 16, dtype, seed=14)
        k_new = torch.randn(33, Hkv, d).to(dtype)
        v_new = torch.randn(33, Hkv, dv).to(dtype)
        cache, _, _, starts = P.cuda(lla)
        lla.lla_paged_append(k_new.cuda(), v_new.cuda(), cache, starts)
        assert lla.lla_stream_status() == 0
        k, v, mass = P.k.clone(), P.v.clone(), P.mass.clone()
        for b, (n, t) in enumerate(zip(P.lens_l, P.news_l)):
            for i in range(t):
                j = n - t + i
                if j >= 0:
                    pg, off = int(P.table[b, j // 16]), j % 16
                    k[pg, :, off], v[pg, :, off] = k_new[P.starts_l[b] + i], v_new[P.starts_l[b] + i]
                    mass[pg, :, off] = 0
        assert torch.equal(cache.k_pages.cpu(), k) and torch.equal(cache.v_pages.cpu(), v)
        assert torch.equal(cache.mass.cpu(), mass)
        # a cache without mass
        bare = lla.PagedCache(P.k.cuda(), P.v.cuda(), P.table.cuda(), P.lens.cuda())
        lla.lla_paged_append(k_new.cuda(), v_new.cuda(), bare, starts)
        assert torch.equal(bare.k_pages.cpu(), k)


def run_evict(lla, P, budget, sinks, recent, max_pages=None):
    cache, _, _, _ = P.cuda(lla)
    B, page = len(P.lens_l), P.page
    counts = [-(-min(n, budget) // page) for n in P.lens_l]
    cap = max_pages or max(1, -(-min(budget, P.table.shape[1] * page) // page))
    table = torch.zeros(B, cap, dtype=torch.int32)
    order = torch.randperm(sum(counts) + 1)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    num = sum(counts) + 1
    to = lla.PagedCache(torch.zeros(num, P.Hkv, page, P.d, dtype=P.dtype, device="cuda"),
                        torch.zeros(num, P.Hkv, page, P.dv, dtype=P.dtype, device="cuda"), table.cuda(),
                        torch.full((B,), -7, dtype=torch.int32, device="cuda"),
                        torch.full((num, P.Hkv, page), -1.0, device="cuda"))
    kept = lla.lla_paged_evict(cache, to, budget, sinks=sinks, recent=recent).cpu()
    assert lla.lla_stream_status() == 0
    ref = evict(P, budget, sinks, recent)
    assert to.lens.cpu().tolist() == [min(n, budget) for n in P.lens_l]
    k, v, mass = torch.zeros_like(to.k_pages).cpu(), torch.zeros_like(to.v_pages).cpu(), to.mass.cpu() * 0 - 1
    for b, n in enumerate(P.lens_l):
        m = min(n, budget)
        pg, off = P.slots(b)
        i = torch.arange(m)
        dp = table[b].long()[i // page]
        for hk in range(P.Hkv):
            assert kept[b, hk].tolist() == ref[b][hk] + [-1] * (budget - m), (b, hk)
            j = torch.tensor(ref[b][hk], dtype=torch.long)
            k[dp, hk, i % page] = P.k[pg[j], hk, off[j]]
            v[dp, hk, i % page] = P.v[pg[j], hk, off[j]]
            mass[dp, hk, i % page] = P.mass[pg[j], hk, off[j]]
    assert torch.equal(to.k_pages.cpu(), k) and torch.equal(to.v_pages.cpu(), v)
    assert torch.equal(to.mass.cpu().nan_to_num(nan=-5.0), mass.nan_to_num(nan=-5.0))


@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 0, 1), (10, 4, 6), (100, 4, 32), (257, 0, 0),
                                                 (5000, 8, 100)])
@pytest.mark.parametrize("dtype,d,dv,Hkv", [(BF, 64, 64, 2), (F32, 16, 32, 1), (F32, 128, 128, 3)])
def test_evict(lla, dtype, d, dv, Hkv, budget, sinks, recent):
    run_evict(lla, Problem([1, 0, 40, 700, 3001, 101], [0] * 6, Hkv, Hkv, d, dv, 16, dtype, seed=15),
              budget, sinks, recent)


def test_evict_ties_and_values_that_are_not_finite(lla):
    P = Problem([600, 2500, 90], [0] * 3, 2, 2, 16, 16, 32, F32, seed=16)
    g = torch.Generator().manual_seed(1)
    levels = torch.tensor([0.0, -0.0, 0.5, 0.5, math.inf, -math.inf, math.nan, 1e-42, -1e-42, -3.0])
    P.mass = levels[torch.randint(0, 10, P.mass.shape, generator=g)]
    for budget in (7, 64, 80, 333, 590, 2499):
        run_evict(lla, P, budget, 3, 4)
    P.mass.zero_()
    run_evict(lla, P, 100, 0, 0)
    P.mass.fill_(math.nan)
    run_evict(lla, P, 100, 2, 2)


def test_evict_long_and_many(lla):
    # a cluster of 8 for one long head; one CTA per head whose keys do not fit shared memory
    run_evict(lla, Problem([20011], [0], 1, 1, 16, 16, 64, F32, seed=17), 5003, 16, 100)
    run_evict(lla, Problem([600] * 20, [0] * 20, 8, 8, 16, 16, 16, F32, seed=18, max_pages=4096), 130, 2, 10)


def test_evict_within_one_pool(lla):
    """Source and destination in the same page arrays, in pages that the source does not hold."""
    P = Problem([100], [0], 1, 1, 16, 16, 16, F32, seed=19, extra_pages=4)
    cache, _, _, _ = P.cuda(lla)
    used = set(P.table[0].tolist())
    free = [x for x in range(P.num_pages) if x not in used]
    to = lla.PagedCache(cache.k_pages, cache.v_pages, torch.tensor([free[:2]], dtype=torch.int32, device="cuda"),
                        torch.zeros(1, dtype=torch.int32, device="cuda"), cache.mass)
    kept = lla.lla_paged_evict(cache, to, 20, sinks=2, recent=3).cpu()
    ref = evict(P, 20, 2, 3)[0][0]
    assert kept[0, 0].tolist() == ref
    pg, off = P.slots(0)
    got = torch.stack([cache.k_pages[free[i // 16], 0, i % 16].cpu() for i in range(20)])
    assert torch.equal(got, P.k[pg[ref], 0, off[ref]])


def test_other_streams_and_graphs(lla):
    """A call on a side stream, and append + attention captured into a graph and replayed."""
    P = Problem([300, 40], [1, 1], 4, 2, 64, 64, 16, BF, True, seed=20)
    ref = attention(P)
    cache, q, r, starts = P.cuda(lla)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, lse = lla.lla_paged_attention(q, cache, starts, P.h, r=r, max_new=1, stream=side)
    side.synchronize()
    check("side stream", out, ref["out"], ref["out_tol"])
    rows = [(P.slots(b)[0][-1], P.slots(b)[1][-1]) for b in range(2)]
    k_new = torch.stack([P.k[pg, :, off] for pg, off in rows]).cuda()
    v_new = torch.stack([P.v[pg, :, off] for pg, off in rows]).cuda()
    out = torch.empty_like(q)
    lse = torch.empty(2, 4, device="cuda")
    n = lla.lla_paged_workspace_size(q, cache, starts, P.h, r=r, max_new=1, track_mass=True, lse=lse)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")

    def step():
        lla.lla_paged_append(k_new, v_new, cache, starts)
        lla.lla_paged_attention(q, cache, starts, P.h, r=r, max_new=1, track_mass=True, out=out, lse=lse,
                                workspace=ws)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for pg, off in rows:
        cache.k_pages[pg, :, off] = 0
    cache.mass.copy_(P.mass)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check("graph", out, ref["out"], ref["out_tol"])


def test_bad_indices_are_reported(lla):
    """What only the device sees: page numbers outside the pool, lengths beyond the table, starts
    that pass the tokens. Nothing is read or written out of range; the status word says so."""
    for dtype, d, news in ((F32, 32, [1, 1]), (BF, 64, [1, 1]), (BF, 128, [40, 1])):
        for what in ("page", "negative page", "length", "negative length", "starts", "descending starts"):
            P = Problem([100, 200], news, 2, 1, d, d, 16, dtype, True, seed=21)
            if "page" in what:
                P.table[0, 3] = -5 if "negative" in what else P.num_pages + 1000
            elif "length" in what:
                P.lens[0] = -1 if "negative" in what else 1 << 29
            else:
                P.starts[1] = P.starts[2] + 5 if what == "starts" else -3
            cache, q, r, starts = P.cuda(lla)
            guard = (cache.k_pages.clone(), cache.v_pages.clone())
            lla.lla_paged_attention(q, cache, starts, P.h, r=r, max_new=max(news), track_mass=True)
            assert lla.lla_stream_status() == 1, what
            assert torch.equal(cache.k_pages, guard[0]) and torch.equal(cache.v_pages, guard[1])
            assert lla.lla_stream_status() == 0
