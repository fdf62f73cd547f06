"""The scratch of paged attention, from its sizes alone (CPU)."""
import ctypes

import pytest

from test_paged_abi import cache, lla, query  # noqa: F401


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("probe", [0, 512])
@pytest.mark.parametrize("max_new,tokens", [(1, 256), (4, 256 * 4), (300, 555)])
def test_scratch_of_weight_tracking_is_bounded(lla, dtype, probe, max_new, tokens):  # noqa: F811
    """The table's capacity sizes the logits that a tracked call keeps: up to two gibibytes of them."""
    def need(pages):
        c = cache(lla, num_seqs=256, kv_heads=8, page_size=1024, max_pages=pages, num_pages=4096, dtype=dtype)
        size = lambda track: lla._load().lla_paged_workspace_size(  # noqa: E731
            ctypes.byref(c), ctypes.byref(query(lla, r=probe or None, lse=4096, tokens=tokens, max_new=max_new, q_heads=64,
                                                track_mass=track)))
        return size(1) - size(0)
    sizes = [need(pages) for pages in (1, 4, 16, 128, 1024, 65535)]
    assert max(sizes) <= 1 << 31 and min(sizes) >= 0, sizes
