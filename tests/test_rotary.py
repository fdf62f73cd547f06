"""Rotary specs and the refusals of lla_rotary and lla_paged_append_rotary, on the CPU: decided on the host, before
any work is enqueued (the pointers are never dereferenced)."""
import ctypes
import math
import struct

import pytest

from test_paged_abi import INVALID, OK, UNSUPPORTED, cache, lla  # noqa: F401


class Spec(ctypes.Structure):
    """lla_rotary_spec, field by field."""
    _fields_ = [("freq", ctypes.c_double * 64), ("scale", ctypes.c_float), ("rot", ctypes.c_int),
                ("layout", ctypes.c_int), ("reserved", ctypes.c_int * 3)]


def spec(**kw):
    s = Spec(scale=1.0, rot=kw.pop("rot", 32), layout=kw.pop("layout", 0))
    for i in range(64):
        s.freq[i] = 0.5 ** i
    for name, value in kw.items():
        if name == "reserved":
            s.reserved[1] = value
        elif name == "freq":
            s.freq[3] = value
        else:
            setattr(s, name, value)
    return s


def frequencies(lla, s, rot=32, layout=0, base=10000.0, stretch=0, factor=1.0, context=0, slow=1.0, fast=32.0):  # noqa: F811
    return lla._load().lla_rotary_frequencies(ctypes.byref(s) if s else None, rot, layout, base, stretch, factor, context,
                                              slow, fast)


def test_struct_size(lla):  # noqa: F811
    assert lla._SPEC.size == ctypes.sizeof(Spec)
    got = Spec.from_buffer_copy(lla._SPEC.pack(*range(64), 2.5, 7, 8, 9, 10, 11))
    assert list(got.freq) == list(range(64)) and got.scale == 2.5
    assert [got.rot, got.layout, *got.reserved] == [7, 8, 9, 10, 11]


@pytest.mark.parametrize("rot", [2, 6, 32, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.0])
def test_frequencies(lla, rot, base):  # noqa: F811
    """Each form from its formula; a power of base is off by a few steps of fp64."""
    near = lambda a, b: abs(a - b) <= 1e-14 * abs(b)  # noqa: E731
    plain = [base ** (-2 * i / rot) for i in range(rot // 2)]
    s = lla.RotarySpec(rot, base=base)
    assert all(map(near, s.freq, plain)) and s.scale == 1 and len(s.freq) == rot // 2
    s = lla.RotarySpec(rot, base=base, stretch=lla.STRETCH_POSITIONS, factor=4.0)
    assert all(near(a, b / 4) for a, b in zip(s.freq, plain))
    if rot > 2:
        s = lla.RotarySpec(rot, base=base, stretch=lla.STRETCH_BASE, factor=4.0)
        assert s.freq[0] == 1 and near(s.freq[-1], plain[-1] / 4)
        assert all(near(a, (base * 4 ** (rot / (rot - 2))) ** (-2 * i / rot)) for i, a in enumerate(s.freq))
    s = lla.RotarySpec(rot, base=base, stretch=lla.STRETCH_WAVELENGTHS, factor=8.0, context=4096, slow=1.0, fast=32.0)
    for a, f in zip(s.freq, plain):
        turns = 4096 * f / (2 * math.pi)
        if turns >= 32:
            assert near(a, f)
        elif turns <= 1:
            assert near(a, f / 8)
        else:
            keep = (turns - 1) / 31
            assert abs(a - f * (keep + (1 - keep) / 8)) <= 1e-13 * f
    assert abs(s.scale - (0.1 * math.log(8) + 1)) <= 2.0 ** -24 * s.scale


def test_a_table_of_ones_own(lla):  # noqa: F811
    s = lla.RotarySpec(6, freq=[1, 0.25, 0], scale=2)
    got = Spec.from_buffer_copy(s._packed)
    assert list(got.freq[:4]) == [1, 0.25, 0, 0] and (got.scale, got.rot, got.layout) == (2, 6, 0)
    for bad in (dict(freq=[1, 2]), dict(freq=[1] * 4)):
        with pytest.raises(ValueError):
            lla.RotarySpec(6, **bad)


@pytest.mark.parametrize("kw", [
    dict(rot=0), dict(rot=3), dict(rot=130), dict(layout=2), dict(layout=-1), dict(base=0.5), dict(base=math.nan),
    dict(base=math.inf), dict(stretch=4), dict(stretch=-1), dict(stretch=1, factor=0.5), dict(stretch=1, factor=math.nan),
    dict(stretch=2, factor=2.0, rot=2), dict(stretch=2, factor=1e300), dict(stretch=3, factor=2.0),
    dict(stretch=3, factor=2.0, context=4096, slow=2.0, fast=2.0),
    dict(stretch=3, factor=2.0, context=4096, slow=math.nan)])
def test_frequency_refusals(lla, kw):  # noqa: F811
    s = spec(scale=7.0)
    before = bytes(s)
    assert frequencies(lla, s, **kw) == INVALID and bytes(s) == before
    assert frequencies(lla, None) == INVALID


def rotate(lla, s, x=(256,), y=None, heads=None, count=None, B=1, T=1, d=64, dtype=1):  # noqa: F811
    y = x if y is None else y
    heads = [2] * len(x) if heads is None else heads
    pack = lambda f, v: struct.pack(f"@{len(v)}{f}", *v)  # noqa: E731
    return lla._load().lla_rotary(ctypes.byref(s) if s else None, pack("P", x), pack("P", y), pack("i", heads),
                                  len(x) if count is None else count, None, B, T, d, 0, dtype, None)


def test_rotary_refusals(lla):  # noqa: F811
    none = dict(T=0)
    assert rotate(lla, spec(), **none) == OK and rotate(lla, spec(), B=0) == OK and rotate(lla, spec(), heads=[0]) == OK
    for bad in (dict(rot=0), dict(rot=66), dict(rot=33), dict(layout=2), dict(reserved=1), dict(freq=math.nan),
                dict(freq=math.inf), dict(freq=2.0 ** 21), dict(scale=math.inf)):
        assert rotate(lla, spec(**bad), **none) == INVALID, bad
    assert rotate(lla, spec(freq=-1.0), **none) == OK
    assert rotate(lla, None, **none) == INVALID
    assert rotate(lla, spec(), count=0) == INVALID and rotate(lla, spec(), x=(256,) * 4, count=4) == INVALID
    assert rotate(lla, spec(), dtype=2) == INVALID and rotate(lla, spec(), B=-1) == INVALID
    assert rotate(lla, spec(), T=-1) == INVALID and rotate(lla, spec(), heads=[-1]) == INVALID
    for d in (8, 48, 256):
        assert rotate(lla, spec(rot=2), d=d) == UNSUPPORTED
    assert rotate(lla, spec(), B=1 << 20, T=1 << 12) == UNSUPPORTED
    assert rotate(lla, spec(), x=(0,)) == INVALID and rotate(lla, spec(), x=(257,)) == INVALID
    assert rotate(lla, spec(), y=(0,)) == INVALID and rotate(lla, spec(), y=(264,)) == INVALID
    assert rotate(lla, spec(), x=(256, 512), y=(1024, 1024)) == INVALID   # written twice
    assert rotate(lla, spec(), x=(256, 512), y=(512, 1024)) == INVALID    # written while read


def append(lla, c=None, s=None, **kw):  # noqa: F811
    f = dict(k=256, v=512, q=768, r=None, q_out=1024, r_out=None, q_heads=4, offsets=None, starts=1280, tokens=4)
    f.update(kw)
    return lla._load().lla_paged_append_rotary(ctypes.byref(c or cache(lla)), ctypes.byref(s or spec()),
                                               *[f[n] for n in ("k", "v", "q", "r", "q_out", "r_out", "q_heads", "offsets",
                                                                "starts", "tokens")], None)


def test_append_refusals(lla):  # noqa: F811
    assert append(lla, tokens=0) == OK and append(lla, c=cache(lla, num_seqs=0)) == OK
    for c, status in ((dict(d=48), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(dtype=2), INVALID),
                      (dict(k_pages=None), INVALID), (dict(lens=None), INVALID)):
        assert append(lla, c=cache(lla, **c)) == status
    assert append(lla, s=spec(rot=66)) == INVALID     # of heads of 64
    assert append(lla, tokens=-1) == INVALID
    assert append(lla, tokens=1 << 30, c=cache(lla, kv_heads=1)) == UNSUPPORTED
    assert append(lla, tokens=1 << 29, q_heads=8, c=cache(lla, kv_heads=1)) == UNSUPPORTED
    for name in ("k", "v", "starts", "q_out"):
        assert append(lla, **{name: None}) == INVALID
    for name in ("k", "v", "q", "q_out"):
        assert append(lla, **{name: 260}) == INVALID
    assert append(lla, q=None, r=256, r_out=512) == INVALID and append(lla, q_heads=0) == INVALID
    assert append(lla, r=2048) == INVALID and append(lla, r=2048, r_out=1024) == INVALID
    assert append(lla, r=2048, r_out=768) == INVALID and append(lla, r=2048, q_out=2048, r_out=4096) == INVALID
