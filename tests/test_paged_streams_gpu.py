"""GPU tests of the paged operators on streams given as objects and as raw handles."""
import pytest
import torch

from paged_reference import Problem
from test_paged_gpu import BF, lla  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True])
def test_streams(lla, raw):  # noqa: F811
    P = Problem([300, 40], [70, 1], 4, 2, 64, 64, 16, BF, True, seed=51)
    cache, q, r, starts = P.cuda(lla)
    out, lse = lla.lla_paged_attention(q, cache, starts, P.h, r=r, max_new=70)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on = side.cuda_stream if raw else side
    k, v = (torch.zeros(71, 2, 64, dtype=BF, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    out2, lse2 = lla.lla_paged_attention(q, cache, starts, P.h, r=r, max_new=70, stream=on)
    lla.lla_paged_append(k, v, cache, starts, stream=on)
    side.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for b in range(2):
        pg, off = P.slots(b)
        new = P.news_l[b]
        assert (cache.k_pages[pg[-new:], :, off[-new:]] == 0).all()
    out3, _ = lla.lla_paged_attention(q, cache, starts, P.h, r=r, max_new=70, stream=0 if raw else torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert lla.lla_stream_status() == 0 and out3.isfinite().all()
