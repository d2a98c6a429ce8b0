"""Refusals of kvq_selftest_tree_timeout that need no GPU."""
import ctypes

import pytest

import quantized_kv_cache_22_b200 as kvq
from test_draft_host import CAPACITY, H, INVALID, LAYER, P, UNSUPPORTED, WINDOW, WORKSPACE, config, ref


def selftest(cfg=None, q=P(16), n=8, max_len=100, wsb=1 << 30, ctas=4, segments=0, limit=1000):
    return kvq.lib().kvq_selftest_tree_timeout(ref(cfg or config()), ref(LAYER), q, 0, n, P(64), max_len, P(128), 0, P(256),
                                               ctypes.c_uint64(wsb), ctas, segments, ctypes.c_uint64(limit), None)


@pytest.mark.parametrize("want,over", [
    (INVALID, dict(limit=0)), (INVALID, dict(limit=2_000_000_001)), (INVALID, dict(segments=-1)), (INVALID, dict(q=None)),
    (INVALID, dict(n=65)), (INVALID, dict(cfg=config(**H))), (UNSUPPORTED, dict(cfg=config(**WINDOW))),
    (CAPACITY, dict(max_len=249)), (WORKSPACE, dict(wsb=16))])
def test_selftest_tree_timeout_refuses(want, over):
    assert selftest(**over) == want
