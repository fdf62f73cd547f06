"""GPU tests of attention of drafted trees against the float64 reference (paged_tree_reference.py)."""
import math

import pytest
import torch

from paged_reference import Problem
from paged_tree_reference import attention, depths, sight, trees
from test_paged_gpu import BF, F32, check, lla  # noqa: F401

pytestmark = pytest.mark.gpu


def flat(forest):
    return torch.tensor([a for tree in forest for a in tree], dtype=torch.int32, device="cuda")


def run(lla, P, forest, window=0, sinks=0, path=0, max_new=None, workspace=False, ref=None):  # noqa: F811
    cache, q, r, starts = P.cuda(lla, mass=False)
    kw = dict(r=r, max_new=max(P.news_l) if max_new is None else max_new, window=window, sinks=sinks, path=path)
    if workspace:
        n = lla.lla_paged_tree_workspace_size(q, cache, starts, P.h, **kw)
        kw["workspace"] = torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda")
    out, lse = lla.lla_paged_tree_attention(q, cache, starts, flat(forest), P.h, **kw)
    assert lla.lla_stream_status() == 0
    ref = ref or attention(P, forest, window, sinks)
    check("out", out, ref["out"], ref["out_tol"])
    check("lse", lse, ref["lse"], ref["lse_tol"])
    return out, lse


# Ragged batches: one node, few rows, several tiles, trees that are all there is, sequences without nodes.
BATCHES = {
    "one": ([1], [1]),
    "single": ([1, 17, 100, 533], [1, 1, 1, 1]),
    "few": ([5, 300, 129, 16], [4, 2, 3, 1]),
    "draft": ([200, 77, 0, 700, 33], [32, 12, 0, 63, 33]),
    "wide": ([400, 150], [260, 7]),
}


@pytest.mark.parametrize("probe", [False, True])
@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("dtype,d,dv,Hq,Hkv,page,branch", [
    (F32, 64, 64, 4, 2, 16, 2), (F32, 16, 128, 3, 1, 64, 3), (BF, 64, 64, 4, 4, 16, 2), (BF, 128, 128, 8, 2, 32, 3),
    (BF, 64, 64, 5, 1, 128, 1), (BF, 128, 128, 21, 3, 256, 4), (BF, 32, 16, 2, 1, 16, 2), (BF, 128, 64, 6, 2, 64, 8),
    (BF, 64, 64, 40, 2, 64, 2), (BF, 64, 32, 12, 4, 32, -1), (F32, 128, 32, 40, 2, 16, 1), (BF, 64, 16, 260, 2, 16, 2)])
def test_tree(lla, dtype, d, dv, Hq, Hkv, page, branch, batch, probe):  # noqa: F811
    lens, news = BATCHES[batch]
    P = Problem(lens, news, Hq, Hkv, d, dv, page, dtype, probe, seed=d + Hq + page)
    run(lla, P, trees(news, branch, seed=Hq))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (3, 500), (7, 3), (64, 130), (300, 5), (10000, 2)])
@pytest.mark.parametrize("batch", ["few", "draft", "wide"])
@pytest.mark.parametrize("dtype,d,probe,branch", [(F32, 32, True, 2), (BF, 64, True, 3), (BF, 128, False, 1),
                                                  (BF, 128, True, 0), (BF, 64, False, 2)])
def test_window_and_sinks(lla, dtype, d, probe, branch, batch, window, sinks):  # noqa: F811
    """The window counts by depth, not by slot: with a deep tree it cuts ancestors off."""
    lens, news = BATCHES[batch]
    run(lla, Problem(lens, news, 6, 2, d, d, 32, dtype, probe, seed=window + sinks), trees(news, branch, 1), window, sinks)


@pytest.mark.parametrize("dtype,d,dv", [(BF, 64, 64), (BF, 128, 128), (F32, 64, 32), (BF, 16, 16)])
@pytest.mark.parametrize("probe", [False, True])
def test_long_sequences_split_over_blocks(lla, dtype, d, dv, probe):  # noqa: F811
    for lens, news in (([9001, 4096, 3], [2, 3, 1]), ([5000], [70])):
        P = Problem(lens, news, 4, 2, d, dv, 64, dtype, probe, seed=5)
        run(lla, P, trees(news, 2), workspace=True)
    P = Problem([3333], [9], 2, 1, d, dv, 16, dtype, probe, seed=7)
    run(lla, P, trees([9], 2), window=2500, sinks=50)


@pytest.mark.parametrize("dtype,d", [(F32, 64), (BF, 64), (BF, 128)])
def test_cuda_core_path(lla, dtype, d):  # noqa: F811
    for batch in ("few", "draft"):
        lens, news = BATCHES[batch]
        run(lla, Problem(lens, news, 6, 2, d, d, 16, dtype, True, seed=11), trees(news, 2), path=1, window=50, sinks=4)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("branch", [0, -1, 3])
def test_a_thousand_nodes(lla, dtype, branch):  # noqa: F811
    P = Problem([1100, 1024], [1023, 1024], 2, 1, 32, 32, 64, dtype, False, seed=2)
    run(lla, P, trees(P.news_l, branch))


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 32)])
@pytest.mark.parametrize("lens,news", [([70], [4]), ([400], [200]), ([9], [9])])
@pytest.mark.parametrize("probe", [False, True])
def test_a_chain_is_the_causal_attention(lla, dtype, d, lens, news, probe):  # noqa: F811
    P = Problem(lens, news, 2, 1, d, d, 16, dtype, probe, seed=8)
    out, lse = run(lla, P, trees(news, 0))
    cache, q, r, starts = P.cuda(lla)
    out2, lse2 = lla.lla_paged_attention(q, cache, starts, P.h, r=r, max_new=news[0])
    ref = attention(P, trees(news, 0))
    check("out", out2, ref["out"], ref["out_tol"])
    check("lse", lse2, ref["lse"], ref["lse_tol"])


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 32)])
@pytest.mark.parametrize("lens,news", [([60], [4]), ([400], [130])])
@pytest.mark.parametrize("probe", [False, True])
@pytest.mark.parametrize("path", [0, 1])
def test_other_branches_may_hold_anything(lla, dtype, d, lens, news, probe, path):  # noqa: F811
    """Node 1's key is NaN and its value infinite: rows that do not go through it come out as without it;
    those that do are not finite. Free pages and the rest of the last one hold junk too."""
    P = Problem(lens, news, 2, 1, d, d, 16, dtype, probe, seed=8)
    forest = trees(news, 2)
    forest[0][1] = -1
    clean = Problem(lens, news, 2, 1, d, d, 16, dtype, probe, seed=8)
    ref = attention(clean, forest)
    pg, off = P.slots(0)
    used = torch.zeros(P.num_pages, 16, dtype=torch.bool)
    used[pg, off] = True
    junk = torch.tensor([math.nan, math.inf, -math.inf, torch.finfo(dtype).max, torch.finfo(dtype).min])
    for x in (P.k, P.v):
        x.copy_(torch.where(used[:, None, :, None], x, junk[torch.arange(d) % 5].to(dtype)))
    at = lens[0] - news[0] + 1
    P.k[pg[at], 0, off[at], 0] = math.nan
    P.v[pg[at], 0, off[at], 1] = math.inf
    cache, q, r, starts = P.cuda(lla, mass=False)
    out, lse = lla.lla_paged_tree_attention(q, cache, starts, flat(forest), P.h, r=r, max_new=news[0], path=path)
    assert lla.lla_stream_status() == 0
    through = sight(lens[0], forest[0], 0, 0)[:, at]
    assert through.any() and not through.all()
    check("out", out[~through.cuda()], ref["out"][~through], ref["out_tol"][~through])
    check("lse", lse[~through.cuda()], ref["lse"][~through], ref["lse_tol"][~through])
    assert out[through.cuda()].isnan().all() and lse[through.cuda()].isnan().all()


@pytest.mark.parametrize("dtype,Hq,t", [(BF, 2, 4), (BF, 4, 60), (F32, 2, 5)])
def test_bad_trees_and_lengths_are_reported(lla, dtype, Hq, t):  # noqa: F811
    """A parent that does not come first, more nodes than positions or than max_new: the other sequence
    comes out right."""
    forest = trees([t, t], 2)
    P = Problem([100, 80], [t, t], Hq, 2, 64, 64, 16, dtype, True, seed=4)
    ref = attention(P, forest)
    for kind in ("parent", "self", "below", "length", "max_new"):
        cache, q, r, starts = P.cuda(lla, mass=False)
        parents = flat(forest)
        n = t
        if kind in ("parent", "self", "below"):
            parents[t + 1] = {"parent": t - 1 if t > 2 else 5, "self": 1, "below": -2}[kind]
        if kind == "length":
            cache.lens[1] = t - 1
        if kind == "max_new":
            cache.lens[0] -= 2
            starts[1:2] -= 2
            n = t - 1
        out, lse = lla.lla_paged_tree_attention(q, cache, starts, parents, P.h, r=r, max_new=n)
        assert lla.lla_stream_status() == 1, kind
        if kind == "max_new":  # the first sequence lost its last two nodes
            assert out[:t - 2].isfinite().all()
            continue
        check("out", out[:t], ref["out"][:t], ref["out_tol"][:t])
        check("lse", lse[:t], ref["lse"][:t], ref["lse_tol"][:t])


def test_rows_that_no_sequence_covers_stay(lla):  # noqa: F811
    for t in (3, 40):
        P = Problem([90, 200], [t, t], 4, 2, 64, 64, 16, BF, False, seed=4)
        cache, q, r, starts = P.cuda(lla, mass=False)
        q = torch.cat([q, q[:5]])
        parents = torch.cat([flat(trees([t, t], 2)), torch.full((5,), 77, dtype=torch.int32, device="cuda")])
        out = torch.full((2 * t + 5, 4, 64), 3.0, dtype=BF, device="cuda")
        lse = torch.full((2 * t + 5, 4), 3.0, device="cuda")
        lla.lla_paged_tree_attention(q, cache, starts, parents, P.h, max_new=t, out=out, lse=lse)
        assert lla.lla_stream_status() == 0
        assert (out[2 * t:] == 3).all() and (lse[2 * t:] == 3).all() and not (out[:2 * t] == 3).all()


@pytest.mark.parametrize("t", [3, 50])
def test_captured_on_another_stream_and_beside_another_call(lla, t):  # noqa: F811
    P = Problem([300, 700], [t, t], 8, 2, 128, 128, 32, BF, False, seed=9)
    forest = trees([t, t], 2)
    cache, q, _, starts = P.cuda(lla, mass=False)
    parents = flat(forest)
    want, want_lse = lla.lla_paged_tree_attention(q, cache, starts, parents, P.h, max_new=t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = lla.lla_paged_tree_attention(q, cache, starts, parents, P.h, max_new=t, stream=side)
    again, _ = lla.lla_paged_tree_attention(q, cache, starts, parents, P.h, max_new=t)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(again, want)
    graph, out, lse = torch.cuda.CUDAGraph(), torch.empty_like(want), torch.empty_like(want_lse)
    with torch.cuda.graph(graph):
        lla.lla_paged_tree_attention(q, cache, starts, parents, P.h, max_new=t, out=out, lse=lse)
        lla.lla_paged_tree_attention(q, cache, starts, parents, P.h, max_new=t, out=out, lse=lse)
    q.mul_(0.5)
    want, want_lse = lla.lla_paged_tree_attention(q, cache, starts, parents, P.h, max_new=t)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert lla.lla_stream_status() == 0


def test_depths_of_the_reference():
    assert depths([-1, 0, 0, 2, -1, 4]) == [0, 1, 1, 2, 0, 1]
