"""Rotary positions, cache and attention without a GPU: refusals at the edges of what is accepted."""
from tests.test_attn_cpu import UNSUPPORTED, _kv, _kv_create


def test_caps_beyond_the_accurate_range_are_refused():
    assert _kv_create(_kv(softcap=2e30)) == UNSUPPORTED
