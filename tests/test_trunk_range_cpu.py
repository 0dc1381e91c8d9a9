"""Refusals at the ends of the trunk operators' ranges, with fake addresses: nothing gets as far as a launch."""
import pytest

from test_trunk_cpu import ab, af, att_desc, lib  # noqa: F401


@pytest.mark.parametrize("scale,refused", [(0.0, False), (1e-45, False), (2.0 ** 127, False), (1.8e38, True), (3e38, True)])
def test_attention_scales(lib, scale, refused):  # noqa: F811
    """A scale times log2(e) has to be a number.  (An accepted call of no queries and keys does nothing.)"""
    assert (af(lib, att_desc(scale=scale, tq=0)) == 3) == refused
    assert (ab(lib, att_desc(scale=scale, tq=0, tk=0)) == 3) == refused
    assert (af(lib, att_desc(scale=scale, tq=0)) == 0) != refused
