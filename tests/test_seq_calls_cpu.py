"""Argument checks of the sequence calls that need no GPU, beside those of test_seq_cpu.py."""
import ctypes

import recsys_feature_interaction_b200 as wk
from tests.test_seq_cpu import FAKE, L, _cache, _cfg, _far  # noqa: F401 (L is a fixture)


def test_a_maximum_of_zero_is_no_way_round_the_checks(L):  # noqa: F811
    c = ctypes.byref(_cfg(max_q=0))
    cache = ctypes.byref(_cache())
    bad = wk.WK_ERR_INVALID_ARG
    assert L.wk_xattn_forward(c, *([None] * 9), 0, None) == bad
    assert L.wk_cache_attention(cache, c, *([None] * 2), None, 4, None, 1, *([None] * 3), 0, None) == bad
    assert L.wk_cache_write(cache, None, None, 0, 0, wk.WK_BF16, None, None, 4, None, 2, 16, 0, None) == bad
    assert L.wk_cache_read(cache, None, 4, None, None, None, None, wk.WK_BF16, 2, 100, 0, None) == bad
