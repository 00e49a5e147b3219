"""Scales belong to an 8-bit cache: attention would apply them and the append would not."""
import pytest

from test_decode_ops_host import P, _append, _attend


@pytest.mark.parametrize("kw", [dict(k_scale=P), dict(v_scale=P), dict(k_scale=P, v_scale=P)])
def test_scales_next_to_a_bf16_cache_are_refused(kw):
    empty = dict(tokens=0), dict(seqs=0)  # calls without work, which are not launched
    assert _append(**kw, **empty[0]) == 4 and _append(**kw, **empty[0], cache_type=2) == 0
    assert _attend(**kw, **empty[1]) == 4 and _attend(**kw, **empty[1], cache_type=2) == 0
