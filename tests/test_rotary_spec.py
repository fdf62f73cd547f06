"""A RotarySpec and the struct that the calls read are one thing: it says what it was made with, and does not change."""
import pytest

from test_paged_abi import lla  # noqa: F401
from test_rotary import Spec


@pytest.mark.parametrize("kw", [dict(), dict(layout=1), dict(freq=[0.5] * 6, scale=2.0, layout=1),
                                dict(stretch=3, factor=4.0, context=512, scale=1.5)])
def test_a_spec_is_what_it_says(lla, kw):  # noqa: F811
    s = lla.RotarySpec(12, **kw)
    packed = Spec.from_buffer_copy(s._packed)
    assert (s.rot, s.layout, s.scale) == (packed.rot, packed.layout, packed.scale) == (12, kw.get("layout", 0), packed.scale)
    assert list(s.freq) == list(packed.freq[:6])


@pytest.mark.parametrize("name,value", [("rot", 8), ("layout", 1), ("scale", 2.0), ("freq", (1.0,) * 6)])
def test_a_spec_does_not_change(lla, name, value):  # noqa: F811
    s = lla.RotarySpec(12)
    before = s._packed, getattr(s, name)
    with pytest.raises(AttributeError):
        setattr(s, name, value)
    assert (s._packed, getattr(s, name)) == before
