"""Argument checks of the sequence calls that need no GPU, beside those of test_seq_cpu.py."""
import ctypes

import recsys_feature_interaction_b200 as wk
from tests.test_seq_cpu import L, _cache, _cfg, _far  # noqa: F401 (L is a fixture)


def test_a_maximum_of_zero_is_no_way_round_the_checks(L):  # noqa: F811
    c = ctypes.byref(_cfg(max_q=0))
    cache = ctypes.byref(_cache())
    bad = wk.WK_ERR_INVALID_ARG
    assert L.wk_xattn_forward(c, *([None] * 9), 0, None) == bad
    assert L.wk_cache_attention(cache, c, *([None] * 2), None, 4, None, 1, *([None] * 3), 0, None) == bad
    assert L.wk_cache_write(cache, None, None, 0, 0, wk.WK_BF16, None, None, 4, None, 2, 16, 0, None) == bad
    assert L.wk_cache_read(cache, None, 4, None, None, None, None, wk.WK_BF16, 2, 100, 0, None) == bad


def test_outputs_over_offsets_lengths_and_tables(L):  # noqa: F811
    """What a launch writes may not lie over the boundaries, lengths and tables that it reads."""
    bad, far = wk.WK_ERR_INVALID_ARG, [_far(i) for i in range(24)]
    c = ctypes.byref(_cfg())
    fwd = [*far[1:4], far[10], far[11], far[12], far[4], far[5], far[6], 1 << 30, None]
    for out in (6, 7):                       # O, lse
        for ints, n in ((3, 3), (4, 3), (5, 2)):
            a = list(fwd)
            a[ints] = a[out] + 16
            assert L.wk_xattn_forward(c, *a) == bad, (out, ints)
            a[ints] = a[out] - 4 * n + 4     # the last value lies in it
            assert L.wk_xattn_forward(c, *a) == bad, (out, ints)
    long = ctypes.byref(_cfg(max_kv=5000))
    a = list(fwd)
    a[3] = a[8] + 64                         # in the workspace
    assert L.wk_xattn_forward(long, *a) == bad
    back = [*far[1:7], far[10], far[11], far[12], *far[7:10], far[13], 1 << 30, None]
    for out in (9, 10, 11, 12):              # dQ, dK, dV, workspace
        for ints in (6, 7, 8):
            a = list(back)
            a[ints] = a[out] + 16
            assert L.wk_xattn_backward(c, *a) == bad, (out, ints)
    cache = ctypes.byref(_cache())           # K, V, exponents at _far(1) .. _far(4)
    write = [far[5], far[6], 0, 0, wk.WK_BF16, far[10], far[11], 4, far[12], 2, 16, 8, None]
    read = [far[11], 4, far[12], far[10], far[5], far[6], wk.WK_BF16, 2, 100, 50, None]
    att = [far[7], far[10], far[11], 4, far[12], 1, far[8], far[9], far[13], 1 << 30, None]
    for held in far[1:5]:
        for ints in (5, 6, 8):
            a = list(write)
            a[ints] = held + 16
            assert L.wk_cache_write(cache, *a) == bad, ints
    for out in (4, 5):
        for ints in (0, 2, 3):
            a = list(read)
            a[ints] = a[out] + 16
            assert L.wk_cache_read(cache, *a) == bad, ints
    for out in (6, 7):
        for ints in (1, 2, 4):
            a = list(att)
            a[ints] = a[out] + 16
            assert L.wk_cache_attention(cache, c, *a) == bad, ints
    a = list(att)
    a[2] = a[6] - 4 * 8 + 4                  # the table's last entry
    assert L.wk_cache_attention(cache, c, *a) == bad
