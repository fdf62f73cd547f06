"""Pages too large for lla_paged_copy's 32-bit counts of 16-byte words, on the CPU: refused on the host, before the device
is asked for anything (the pointers are never dereferenced)."""
import ctypes

import pytest

from test_paged_abi import UNSUPPORTED, cache, lla  # noqa: F401


def copy(lla, count=1, **kw):  # noqa: F811
    c = ctypes.byref(cache(lla, num_pages=2, **kw))
    return lla._load().lla_paged_copy(c, c, 256, count, None)


@pytest.mark.parametrize("kw", [
    dict(dtype=0, kv_heads=65535, page_size=1024, d=64, dv=64),  # 2^30 - 2^14 words each of keys and values, 2^24 of mass
    dict(dtype=0, kv_heads=65535, page_size=1024, d=128, dv=128, mass=None)])
def test_pages_beyond_32_bits(lla, kw):  # noqa: F811
    assert kw["kv_heads"] * kw["page_size"] * ((kw["d"] + kw["dv"]) * 4 + 4 * ("mass" not in kw)) // 16 >= 2 ** 31
    assert copy(lla, **kw) == UNSUPPORTED


def test_many_pairs(lla):  # noqa: F811
    assert copy(lla, page_size=1024, count=1 << 30) == UNSUPPORTED
