"""GPU tests of fp32 attention over a paged cache where its kernel changes form: rows to a tile, tiles to
a token, splits joined in a cluster or through scratch, and where the weights come from."""
import pytest
import torch

from paged_reference import Problem
from test_paged_gpu import F32, lla, run_and_check  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("probe", [False, True])
@pytest.mark.parametrize("g", [1, 3, 4, 5, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("d,dv", [(128, 128), (64, 64), (32, 128), (128, 16)])
def test_rows_of_a_tile(lla, d, dv, g, probe):  # noqa: F811
    news = [1, 2, 3, 5]
    run_and_check(lla, Problem([33, 31, 70, 5], news, 2 * g, 2, d, dv, 16, F32, probe, seed=g))


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (15, 17), (90, 3), (333, 40)])
@pytest.mark.parametrize("g", [1, 5, 16])
def test_many_tiles_with_a_window(lla, g, window, sinks):  # noqa: F811
    run_and_check(lla, Problem([500, 47, 1, 300], [16, 15, 1, 1], g, 1, 128, 64, 32, F32, True, seed=window), window, sinks)


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5)])
def test_weights_of_long_chunks_beside_single_tokens(lla, window, sinks):  # noqa: F811
    run_and_check(lla, Problem([700, 400, 9], [300, 1, 2], 4, 2, 64, 64, 64, F32, False, seed=1), window, sinks)


def test_weights_where_the_table_has_room_for_many_more_positions(lla):  # noqa: F811
    run_and_check(lla, Problem([700, 40, 2000], [30, 1, 9], 4, 2, 32, 32, 1024, F32, True, seed=2, max_pages=400))


@pytest.mark.parametrize("probe", [False, True])
@pytest.mark.parametrize("n", [1, 40])
def test_more_splits_than_a_cluster_has(lla, n, probe):  # noqa: F811
    run_and_check(lla, Problem([15001], [n], 3, 1, 64, 128, 16, F32, probe, seed=3), workspace=True)


def test_rows_of_one_batch_need_different_references(lla):  # noqa: F811
    """Maxima that grow along the keys, by more and by less than the reference may lag."""
    P = Problem([900, 900], [1, 20], 4, 1, 64, 64, 16, F32, True, seed=4)
    for b in range(2):
        pg, off = P.slots(b)
        P.k[pg, :, off] *= torch.linspace(0.01, 12.0, 900)[:, None, None]
    run_and_check(lla, P)
