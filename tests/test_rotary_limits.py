"""Head counts near 2^31, on the CPU: refused on the host before the device is asked for anything (the pointers are never
dereferenced). With a few fewer the last ones would fall out of the launch's 31-bit indices."""
from test_paged_abi import OK, UNSUPPORTED, lla  # noqa: F401
from test_rotary import append, rotate, spec


def test_rotary(lla):  # noqa: F811
    most = 2 ** 31 - 2 ** 17
    assert rotate(lla, spec(), heads=[2 ** 31 - 1]) == UNSUPPORTED
    assert rotate(lla, spec(), heads=[most + 1]) == UNSUPPORTED
    assert rotate(lla, spec(), x=(256, 512, 768), heads=[most, 1, 0]) == UNSUPPORTED
    assert rotate(lla, spec(), heads=[most], T=0) == OK


def test_append(lla):  # noqa: F811
    kw = dict(tokens=1, r=2048, r_out=4096)
    for heads in (2 ** 30, 2 ** 31 - 1, 2 ** 30 - 2 ** 16):  # of q and of r
        assert append(lla, q_heads=heads, **kw) == UNSUPPORTED
    assert append(lla, q_heads=2 ** 31 - 1, tokens=1) == UNSUPPORTED
