"""GPU tests of trees below contexts long enough for the tensor-core kernel with few rows: key tiles in pairs (heads of
128, softmax, at most 128 rows) with odd numbers of tiles, shares that cut tiles, windows, slots that hold
anything and logits that outgrow their reference."""
import math

import pytest
import torch

from paged_reference import Problem
from paged_tree_reference import attention, sight, trees
from test_paged_gpu import BF, check, lla  # noqa: F401
from test_paged_tree_gpu import flat, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,probe", [(128, False), (128, True), (64, False), (64, True)])
@pytest.mark.parametrize("lens,news", [([9000], [40]), ([8193, 130, 4000], [33, 64, 60]), ([300, 12001], [64, 50])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2100, 9)])
def test_few_rows_long_context(lla, d, probe, lens, news, window, sinks):  # noqa: F811
    P = Problem(lens, news, 8, 4, d, d, 32, BF, probe, seed=len(lens), max_pages=400)
    run(lla, P, trees(news, 2, 3), window, sinks)


@pytest.mark.parametrize("dv,page,g", [(128, 128, 2), (16, 16, 3), (128, 256, 1)])
def test_pairs_of_key_tiles(lla, dv, page, g):  # noqa: F811
    """One, two and three tiles to a tree, and pieces of any number of them."""
    lens, news = [40, 129, 257, 1025, 6000, 64], [40, 42, 36, 41, 42, 1]
    P = Problem(lens, news, 2 * g, 2, 128, dv, page, BF, False, seed=dv, max_pages=40000 // page)
    run(lla, P, trees(news, 3, 1), workspace=True)


def test_more_sequences_than_ctas(lla):  # noqa: F811
    lens = [200 + 37 * b for b in range(100)]
    P = Problem(lens, [36] * 100, 2, 2, 128, 128, 64, BF, False, seed=3)
    run(lla, P, trees([36] * 100, 2, 5))


@pytest.mark.parametrize("at", [-1, 200, 8100])
def test_values_in_hidden_slots(lla, at):  # noqa: F811
    """A position that fell out of the window (or, at -1, another branch) holds NaN and infinity."""
    lens, news, window = [9000], [50], 600
    P = Problem(lens, news, 8, 4, 128, 128, 32, BF, False, seed=9, max_pages=400)
    forest = trees(news, 2, 2)
    forest[0][1] = -1
    ref = attention(P, forest, window, 5)
    pg, off = P.slots(0)
    slot = lens[0] - news[0] + 1 if at < 0 else at
    P.k[pg[slot], :, off[slot]] = math.nan
    P.v[pg[slot], :, off[slot]] = math.inf
    cache, q, _, starts = P.cuda(lla, mass=False)
    out, lse = lla.lla_paged_tree_attention(q, cache, starts, flat(forest), P.h, max_new=50, window=window, sinks=5)
    assert lla.lla_stream_status() == 0
    hidden = ~sight(lens[0], forest[0], window, 5)[:, slot]
    assert hidden.any() and (at < 0 or hidden.all())
    check("out", out[hidden.cuda()], ref["out"][hidden], ref["out_tol"][hidden])
    check("lse", lse[hidden.cuda()], ref["lse"][hidden], ref["lse_tol"][hidden])


@pytest.mark.parametrize("where", [5, 130, 3000, 8999])
def test_a_key_that_outgrows_the_others(lla, where):  # noqa: F811
    """One key's logits are far above the others': in the first tile of a stream, in its second, late, and a node's own."""
    lens, news = [9000], [50]
    P = Problem(lens, news, 8, 4, 128, 128, 32, BF, False, seed=4, max_pages=400)
    pg, off = P.slots(0)
    P.k[pg[where], :, off[where]] = P.k[pg[where], :, off[where]] * 40
    run(lla, P, trees(news, 0))


def test_the_same_bits_whatever_the_run(lla):  # noqa: F811
    P = Problem([9000, 700, 5000], [50, 64, 33], 8, 4, 128, 128, 32, BF, False, seed=4, max_pages=400)
    forest = trees(P.news_l, 2)
    cache, q, _, starts = P.cuda(lla, mass=False)
    first = lla.lla_paged_tree_attention(q, cache, starts, flat(forest), P.h, max_new=64)
    for _ in range(5):
        again = lla.lla_paged_tree_attention(q, cache, starts, flat(forest), P.h, max_new=64)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("d,t", [(128, 50), (64, 70), (128, 200)])
def test_two_streams_and_a_graph_with_one_workspace(lla, d, t):  # noqa: F811
    P = Problem([9000, 4100], [t, t], 8, 4, d, d, 32, BF, False, seed=6, max_pages=400)
    cache, q, _, starts = P.cuda(lla, mass=False)
    parents = [flat(trees(P.news_l, branch, 1)) for branch in (2, 0)]
    call = lambda i, **kw: lla.lla_paged_tree_attention(q, cache, starts, parents[i], P.h, max_new=t, **kw)  # noqa: E731
    want = [call(i) for i in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [(call(0), call(1, stream=side)) for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        for i in range(2):
            assert torch.equal(pair[i][0], want[i][0]) and torch.equal(pair[i][1], want[i][1])
    size = lla.lla_paged_tree_workspace_size(q, cache, starts, P.h, max_new=t)
    workspace = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    outs = [(torch.empty_like(o), torch.empty_like(x)) for o, x in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i, (o, x) in enumerate(outs):
            call(i, out=o, lse=x, workspace=workspace)
    q.mul_(0.5)
    for _ in range(3):
        graph.replay()
    want = [call(i) for i in range(2)]
    torch.cuda.synchronize()
    for (o, x), (a, b) in zip(outs, want):
        assert torch.equal(o, a) and torch.equal(x, b)
    assert lla.lla_stream_status() == 0


def test_a_node_without_anything_to_see(lla):  # noqa: F811
    """Roots with no context before them whose own logit is -infinity: nothing comes out of them, their children
    see themselves."""
    for dtype, d in ((BF, 128), (BF, 64), (torch.float32, 32)):
        P = Problem([40], [40], 2, 1, d, d, 16, dtype, False, seed=2)
        forest = [[-1] * 20 + list(range(20))]
        pg, off = P.slots(0)
        P.q[:] = P.q.abs()
        P.k[pg[:20], :, off[:20]] = -math.inf
        cache, q, _, starts = P.cuda(lla, mass=False)
        out, lse = lla.lla_paged_tree_attention(q, cache, starts, flat(forest), P.h, max_new=40)
        assert lla.lla_stream_status() == 0
        assert (out[:20] == 0).all() and (lse[:20] == -math.inf).all()
        own = P.v[pg[20:], 0, off[20:]].to(torch.float64)[:, None].expand(-1, 2, -1)
        check("out", out[20:], own, own.abs() * (2.0 ** -8 if dtype == BF else 2.0 ** -22))
