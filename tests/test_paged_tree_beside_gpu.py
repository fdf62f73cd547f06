"""GPU test of trees beside one that has more nodes than max_new: that one is reported and written nowhere else, the others
come out right. Outputs begin as NaN, so that a row that is not computed shows. References and bounds as in
test_paged_tree_gpu.py."""
import math

import pytest
import torch

from paged_reference import Problem
from paged_tree_reference import attention, trees
from test_paged_gpu import BF, F32, check, lla  # noqa: F401
from test_paged_tree_gpu import flat

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("big", [0, 1, 2])
@pytest.mark.parametrize("dtype,Hq,Hkv,d,probe,path,max_new,beyond", [
    (BF, 4, 2, 64, True, 0, 2, 3),          # a tile of few rows
    (BF, 4, 2, 128, False, 0, 4, 9),
    (BF, 2, 2, 64, True, 0, 60, 61),        # tiles of few rows
    (BF, 8, 2, 64, False, 0, 60, 64),       # the tensor-core kernels, beside few rows and alone
    (BF, 4, 4, 128, False, 0, 100, 101),
    (BF, 16, 4, 128, False, 0, 200, 260),
    (BF, 4, 2, 128, True, 0, 150, 151),
    (BF, 4, 2, 64, True, 1, 30, 31),        # CUDA cores
    (F32, 4, 2, 64, True, 0, 5, 6),
    (F32, 2, 2, 128, False, 0, 64, 65),
    (F32, 2, 1, 32, True, 0, 100, 170)])
def test_more_nodes_than_max_new(lla, dtype, Hq, Hkv, d, probe, path, max_new, beyond, big):  # noqa: F811
    news = [max_new, 1, max(1, max_new - 3)]
    news[big] = beyond
    lens = [700, 300, 901]
    P = Problem(lens, news, Hq, Hkv, d, d, 16, dtype, probe, seed=beyond)
    forest = trees(news, 2)
    ref = attention(P, forest)
    cache, q, r, starts = P.cuda(lla, mass=False)
    out = torch.full((sum(news), Hq, d), math.nan, dtype=dtype, device="cuda")
    lse = torch.full((sum(news), Hq), math.nan, device="cuda")
    lla.lla_paged_tree_attention(q, cache, starts, flat(forest), P.h, r=r, max_new=max_new, path=path, out=out, lse=lse)
    assert lla.lla_stream_status() == 1
    for b in range(3):
        if b != big:
            rows = slice(sum(news[:b]), sum(news[:b + 1]))
            check("out", out[rows], ref["out"][rows], ref["out_tol"][rows])
            check("lse", lse[rows], ref["lse"][rows], ref["lse_tol"][rows])
