"""Attention over behaviour sequences without a GPU: the oracle's functions pinned by identities and
differences, the index arithmetic's answers to broken offsets, lengths and tables, and the refusals
of the C entry points and the binding."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import oracle
import recsys_feature_interaction_b200 as wk

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    from recsys_feature_interaction_b200 import build
    build.build()
    return wk.lib()


# ------------------------------------------------------------------------------ oracle

def test_one_key_is_its_value():
    r = np.random.RandomState(0)
    q, k, v = r.randn(3, 4, 8), r.randn(1, 2, 8), r.randn(1, 2, 8)
    O, lse = oracle.sequence_attention(q, k, v)
    assert np.allclose(O, np.repeat(np.repeat(v, 2, axis=1), 3, axis=0))
    assert np.allclose(lse[:, 0], (q[:, 0] * k[0, 0]).sum(-1) / np.sqrt(8))


def test_shared_keys_give_the_module_attention():
    r = np.random.RandomState(1)
    q, k = r.randn(5, 1, 16), r.randn(9, 1, 16)
    O, _ = oracle.sequence_attention(q, k, k)
    assert np.allclose(O[:, 0], oracle.attention_shared_kv(q[:, 0], k[:, 0]))


def test_newest_rows_see_their_past():
    r = np.random.RandomState(2)
    q, k, v = r.randn(4, 2, 8), r.randn(6, 1, 8), r.randn(6, 1, 8)
    O, lse = oracle.sequence_attention(q, k, v, new_rows=4)
    for i in range(4):
        o, l = oracle.sequence_attention(q[i:i + 1], k[:3 + i], v[:3 + i])
        assert np.allclose(O[i], o[0]) and np.allclose(lse[i], l[0])
    O, lse = oracle.sequence_attention(q, k[:2], v[:2], new_rows=4)
    assert (O[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2:]).all()


def test_gradients_by_differences():
    r = np.random.RandomState(3)
    ten = [r.randn(4, 4, 6), r.randn(5, 2, 6), r.randn(5, 2, 6)]
    dO = r.randn(4, 4, 6)
    grads = oracle.sequence_attention_backward(*ten, dO)
    for i in range(3):
        step = r.randn(*ten[i].shape)
        f = []
        for h in (1e-6, -1e-6):
            a = list(ten)
            a[i] = ten[i] + h * step
            f.append((oracle.sequence_attention(*a)[0] * dO).sum())
        assert abs((f[0] - f[1]) / 2e-6 - (grads[i] * step).sum()) < 1e-7
    for g, t in zip(oracle.sequence_attention_backward(ten[0], ten[1][:0], ten[2][:0], dO), ten):
        assert (g == 0).all()


def test_e4m3_rounding_matches_the_type():
    x = np.random.RandomState(4).uniform(-448, 448, 20000)
    x[:6000] *= 1e-3
    x = x.astype(np.float32)  # the type's own conversion starts from fp32
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.e4m3_round(x), ref)


def test_quantised_rows():
    rows = np.array([[0.0, 0.0], [448.0, 1.0], [448.5, 1.0], [2.0 ** -120, 0.0], [np.inf, 1.0], [1.0, np.nan]])
    v, e = oracle.cache_quantise(rows)
    assert list(e) == [0, 127, 128, 0, 255, 255]
    assert np.array_equal(v[0], [0, 0]) and np.array_equal(v[1], [448, 1]) and np.array_equal(v[2], [224, 0.5])
    assert v[3][0] == 128.0 and np.isnan(v[4]).all() and np.isnan(v[5]).all()
    r = np.random.RandomState(5).randn(50, 32) * np.exp(np.random.RandomState(6).randn(50, 1) * 5)
    v, e = oracle.cache_quantise(r)
    amax = np.abs(v).max(axis=1)
    assert (amax <= 448).all() and (amax > 200).all()  # the least power: more than half the range is used
    back = v * np.ldexp(1.0, e.astype(int) - 127)[:, None]
    step = np.ldexp(1.0, e.astype(int) - 127)[:, None]
    assert (np.abs(back - r) <= np.maximum(np.abs(r) * 2.0 ** -4, step * 2.0 ** -10)).all()


# -------------------------------------------------------------- index arithmetic, broken tables

@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_index_arithmetic_stays_inside(tmp_path):
    exe = str(tmp_path / "check")
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I",
                        os.path.join(ROOT, "recsys_feature_interaction_b200", "csrc"),
                        os.path.join(ROOT, "tests", "c_abi", "seq_index_check.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    asked, want = [], []

    def ask(line, answer):
        asked.append(line)
        want.append(answer)

    # lo hi len total most -> begin len room bad
    ask("span 3 10 -99 20 16", "3 7 7 0")
    ask("span 3 10 4 20 16", "3 4 7 0")
    ask("span 3 3 -99 20 16", "3 0 0 0")
    ask("span 0 30 -99 20 64", "0 20 20 1")     # past the tensor
    ask("span 25 30 -99 20 64", "20 0 0 1")     # begins behind it
    ask("span -4 5 -99 20 64", "0 5 5 1")
    ask("span 9 2 -99 20 64", "9 0 0 1")        # decreasing
    ask("span 3 10 8 20 16", "3 7 7 1")         # more keys than room
    ask("span 3 10 -1 20 16", "3 0 7 1")
    ask("span 3 10 -99 20 5", "3 5 7 1")        # longer than the caller said
    ask("span -2147483648 2147483647 -99 20 64", "0 20 20 1")
    ask("cached 100 128 200 0 0", "0 100 100 0")
    ask("cached 129 128 200 0 0", "0 128 128 1")
    ask("cached 100 128 90 0 0", "0 90 90 1")
    ask("cached -3 128 90 0 0", "0 0 0 1")
    ask("page 7 100 4 9 0", "7")
    ask("page 9 100 4 9 0", "-1")
    ask("page -1 100 4 9 0", "-1")
    ask("page 2147483647 1000 4 9 0", "-1")
    ask("seen 10 4 0 1 0", "7")
    ask("seen 10 4 3 1 0", "10")
    ask("seen 10 4 0 0 0", "10")
    ask("seen 2 5 2 1 0", "0")
    ask("seen 2 5 3 1 0", "1")
    ask("seen 0 1 0 1 0", "0")
    out = subprocess.run([exe], input="\n".join(asked) + "\n", capture_output=True, text=True).stdout.splitlines()
    assert out == want


# ------------------------------------------------------------------------------ refusals

FAKE = 1 << 20


def _cfg(**kw):
    c = dict(batch=2, q_heads=4, kv_heads=2, d=64, max_q=8, max_kv=100, total_q=16, total_kv=150, q_stride=0,
             k_stride=0, v_stride=0, dtype=wk.WK_BF16, scale=0.0)
    c.update(kw)
    return wk.WkXattnConfig(*[c[f[0]] for f in wk.WkXattnConfig._fields_])


BAD_CONFIG = [
    (dict(batch=-1), wk.WK_ERR_INVALID_ARG), (dict(q_heads=0), wk.WK_ERR_INVALID_ARG),
    (dict(kv_heads=3), wk.WK_ERR_INVALID_ARG), (dict(d=96), wk.WK_ERR_UNSUPPORTED),
    (dict(dtype=wk.WK_F32), wk.WK_ERR_UNSUPPORTED), (dict(dtype=wk.WK_E4M3), wk.WK_ERR_UNSUPPORTED),
    (dict(max_q=-1), wk.WK_ERR_INVALID_ARG), (dict(total_q=-1), wk.WK_ERR_INVALID_ARG),
    (dict(total_kv=1 << 50), wk.WK_ERR_INVALID_ARG), (dict(q_stride=100), wk.WK_ERR_INVALID_ARG),
    (dict(k_stride=132), wk.WK_ERR_UNSUPPORTED), (dict(v_stride=-128), wk.WK_ERR_INVALID_ARG),
    (dict(scale=-1.0), wk.WK_ERR_INVALID_ARG), (dict(scale=float("nan")), wk.WK_ERR_INVALID_ARG),
    (dict(scale=float("inf")), wk.WK_ERR_INVALID_ARG), (dict(q_heads=2048, kv_heads=2048), wk.WK_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("bad,status", BAD_CONFIG)
def test_configs_that_are_refused(L, bad, status):
    c = _cfg(**bad)
    n = ctypes.c_int64(7)
    assert L.wk_xattn_workspace(ctypes.byref(c), 1, ctypes.byref(n)) == status and n.value == 7
    p = [FAKE << i for i in range(12)]
    assert L.wk_xattn_forward(ctypes.byref(c), *p[:3], FAKE, FAKE, None, p[5], None, p[6], 1 << 40, None) == status
    assert L.wk_xattn_backward(ctypes.byref(c), *p[:4], FAKE, p[5], FAKE, FAKE, None, *p[6:9], p[9], 1 << 40,
                               None) == status


def _far(i):
    return FAKE + (i << 32)


def test_pointers_that_are_refused(L):
    c = _cfg()
    good = [_far(1), _far(2), _far(3), FAKE, FAKE, None, _far(4), None, _far(5), 1 << 30, None]

    def call(**kw):
        a = list(good)
        for i, x in kw.items():
            a[int(i[1:])] = x
        return L.wk_xattn_forward(ctypes.byref(c), *a)

    for i in (0, 1, 2, 3, 4, 6):
        assert call(**{"a%d" % i: None}) == wk.WK_ERR_INVALID_ARG
    for i in (0, 1, 2, 6, 8):
        assert call(**{"a%d" % i: good[i] + 8}) == wk.WK_ERR_INVALID_ARG
    for i in (3, 4, 5, 7):
        assert call(**{"a%d" % i: FAKE + 2}) == wk.WK_ERR_INVALID_ARG
    assert call(a6=_far(1) + 64) == wk.WK_ERR_INVALID_ARG       # O over Q
    assert call(a6=_far(2)) == wk.WK_ERR_INVALID_ARG            # O over K
    assert call(a7=_far(4) + 16) == wk.WK_ERR_INVALID_ARG       # lse in O
    assert call(a7=_far(1)) == wk.WK_ERR_INVALID_ARG            # lse over Q
    assert L.wk_xattn_forward(ctypes.byref(_cfg(max_kv=5000)), *(good[:8] + [_far(2)] + good[9:])) \
        == wk.WK_ERR_INVALID_ARG                                # the workspace over K
    assert call(a9=-1) == wk.WK_ERR_INVALID_ARG
    e = _cfg(batch=0)
    assert L.wk_xattn_forward(ctypes.byref(e), *([None] * 9), 0, None) == wk.WK_OK
    e = _cfg(total_q=0)
    assert L.wk_xattn_forward(ctypes.byref(e), *([None] * 9), 0, None) == wk.WK_OK
    # the backward: too small a workspace, gradients over inputs or one another
    back = [_far(1), _far(2), _far(3), _far(4), _far(5), _far(6), FAKE, FAKE, None, _far(7), _far(8), _far(9), _far(10),
            1 << 30, None]
    n = ctypes.c_int64()
    assert L.wk_xattn_workspace(ctypes.byref(c), 1, ctypes.byref(n)) == wk.WK_OK and n.value > 0

    def grad(i, x):
        a = list(back)
        a[i] = x
        return L.wk_xattn_backward(ctypes.byref(c), *a)

    assert grad(13, n.value - 1) == wk.WK_ERR_INVALID_ARG
    assert grad(12, None) == wk.WK_ERR_INVALID_ARG
    assert grad(9, _far(1)) == wk.WK_ERR_INVALID_ARG and grad(10, _far(3) + 256) == wk.WK_ERR_INVALID_ARG
    assert grad(12, _far(5)) == wk.WK_ERR_INVALID_ARG           # the workspace over dO
    assert grad(11, _far(8)) == wk.WK_ERR_INVALID_ARG and grad(9, _far(10)) == wk.WK_ERR_INVALID_ARG
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 9, 10, 11):
        assert grad(i, None) == wk.WK_ERR_INVALID_ARG


def _cache(**kw):
    c = dict(K=_far(1), V=_far(2), K_exp=_far(3), V_exp=_far(4), num_pages=10, page_size=16, kv_heads=2, d=64,
             dtype=wk.WK_E4M3)
    c.update(kw)
    return wk.WkCache(*[c[f[0]] for f in wk.WkCache._fields_])


@pytest.mark.parametrize("bad,status", [
    (dict(page_size=48), wk.WK_ERR_UNSUPPORTED), (dict(page_size=256), wk.WK_ERR_UNSUPPORTED),
    (dict(d=96), wk.WK_ERR_UNSUPPORTED), (dict(dtype=wk.WK_F32), wk.WK_ERR_UNSUPPORTED),
    (dict(K=_far(1) + 8), wk.WK_ERR_INVALID_ARG), (dict(K_exp=None), wk.WK_ERR_INVALID_ARG),
    (dict(V_exp=_far(4) + 1), wk.WK_ERR_INVALID_ARG), (dict(V=None), wk.WK_ERR_INVALID_ARG),
    (dict(dtype=wk.WK_BF16), wk.WK_ERR_INVALID_ARG),  # exponents with a 16-bit cache
    (dict(num_pages=-1), wk.WK_ERR_INVALID_ARG), (dict(kv_heads=0), wk.WK_ERR_INVALID_ARG)])
def test_caches_that_are_refused(L, bad, status):
    c = _cache(**bad)
    r = ctypes.byref(c)
    cfg = _cfg(d=c.d if c.d in (32, 64, 128, 160) else 64, kv_heads=max(1, c.kv_heads))
    n = ctypes.c_int64()
    assert L.wk_cache_write(r, _far(5), _far(6), 0, 0, wk.WK_BF16, FAKE, FAKE, 4, FAKE, 2, 16, 8, None) == status
    assert L.wk_cache_read(r, FAKE, 4, FAKE, FAKE, _far(5), _far(6), wk.WK_BF16, 2, 100, 50, None) == status
    assert L.wk_cache_attention_workspace(r, ctypes.byref(cfg), ctypes.byref(n)) == status
    assert L.wk_cache_attention(r, ctypes.byref(cfg), _far(7), FAKE, FAKE, 4, FAKE, 1, _far(8), None, _far(9), 1 << 30,
                                None) == status


def test_cache_calls_that_are_refused(L):
    q8, q16 = _cache(), _cache(K_exp=None, V_exp=None, dtype=wk.WK_F16)
    w = [_far(5), _far(6), 0, 0, wk.WK_BF16, FAKE, FAKE, 4, FAKE, 2, 16, 8, None]

    def write(c, **kw):
        a = list(w)
        for i, x in kw.items():
            a[int(i[1:])] = x
        return L.wk_cache_write(ctypes.byref(c), *a)

    assert write(q16) == wk.WK_ERR_UNSUPPORTED              # bf16 tokens, fp16 cache
    assert write(q8, a4=wk.WK_F32) == wk.WK_ERR_UNSUPPORTED
    assert write(q8, a2=64) == wk.WK_ERR_INVALID_ARG and write(q8, a2=132) == wk.WK_ERR_UNSUPPORTED
    assert write(q8, a9=-1) == wk.WK_ERR_INVALID_ARG and write(q8, a9=0) == wk.WK_OK
    assert write(q8, a7=0) == wk.WK_ERR_INVALID_ARG and write(q8, a10=0) == wk.WK_OK
    for i in (0, 1, 5, 6, 8):
        assert write(q8, **{"a%d" % i: None}) == wk.WK_ERR_INVALID_ARG
        assert write(q8, **{"a%d" % i: FAKE + 2}) == wk.WK_ERR_INVALID_ARG
    n = ctypes.c_int64()
    for c, cfg, status in ((q8, _cfg(d=128), wk.WK_ERR_INVALID_ARG), (q8, _cfg(kv_heads=1), wk.WK_ERR_INVALID_ARG),
                           (q16, _cfg(), wk.WK_ERR_UNSUPPORTED)):
        assert L.wk_cache_attention_workspace(ctypes.byref(c), ctypes.byref(cfg), ctypes.byref(n)) == status
    r = [FAKE, 4, FAKE, FAKE, _far(5), _far(6), wk.WK_BF16, 2, 100, 50, None]
    assert L.wk_cache_read(ctypes.byref(q8), *(r[:5] + [_far(5) + 128] + r[6:])) == wk.WK_ERR_INVALID_ARG  # V over K
    assert L.wk_cache_read(ctypes.byref(q16), *r) == wk.WK_ERR_UNSUPPORTED
    # buffers that lie over one another
    assert write(_cache(V=_far(1) + 64)) == wk.WK_ERR_INVALID_ARG
    assert write(q8, a0=_far(1)) == wk.WK_ERR_INVALID_ARG and write(q8, a1=_far(1) + 128) == wk.WK_ERR_INVALID_ARG
    assert L.wk_cache_read(ctypes.byref(q8), *(r[:4] + [_far(2)] + r[5:])) == wk.WK_ERR_INVALID_ARG
    assert write(_cache(K_exp=_far(1) + 64)) == wk.WK_ERR_INVALID_ARG
    cfg = _cfg()
    att = [_far(7), FAKE, FAKE, 4, FAKE, 1, _far(8), None, _far(9), 1 << 30, None]
    assert L.wk_cache_attention(ctypes.byref(q8), ctypes.byref(cfg), *(att[:7] + [_far(7)] + att[8:])) \
        == wk.WK_ERR_INVALID_ARG  # lse over Q
    for over in (_far(7) + 32, _far(1) + 16, _far(2), _far(4)):
        assert L.wk_cache_attention(ctypes.byref(q8), ctypes.byref(cfg), *(att[:6] + [over] + att[7:])) \
            == wk.WK_ERR_INVALID_ARG


def test_the_binding_refuses(L):
    """Shapes, types and devices are looked at before the library is called."""
    q, k = torch.zeros(6, 4, 64, dtype=torch.bfloat16), torch.zeros(9, 2, 64, dtype=torch.bfloat16)
    off, koff = torch.tensor([0, 6], dtype=torch.int32), torch.tensor([0, 9], dtype=torch.int32)

    def forward(**kw):
        a = dict(Q=q, K=k, V=k, O=torch.zeros_like(q), q_off=off, kv_off=koff, max_q=6, max_kv=9)
        a.update(kw)
        wk.wk_xattn_forward(**a)

    for bad in (dict(), dict(K=k.half()), dict(K=k[:, :, :32]), dict(V=k[:5]), dict(q_off=off.long()),
                dict(kv_off=torch.tensor([0, 1, 9], dtype=torch.int32)), dict(O=torch.zeros(6, 4, 32)),
                dict(Q=q.transpose(0, 1)), dict(K=k[:1].expand(9, 2, 64)), dict(lse=torch.zeros(6, 4, dtype=torch.float64)),
                dict(kv_lens=torch.zeros(2, dtype=torch.int32)), dict(O=torch.zeros(6, 64, 4).transpose(1, 2))):
        with pytest.raises(ValueError):  # the first one: nothing wrong but the device
            forward(**bad)
    c8 = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    e8 = torch.zeros(4, 2, 16, dtype=torch.uint8)
    for bad in (dict(K=c8, V=c8), dict(K=c8, V=c8, K_exp=e8, V_exp=e8[:2]), dict(K=c8, V=c8[:2], K_exp=e8, V_exp=e8),
                dict(K=c8.bool(), V=c8.bool(), K_exp=e8, V_exp=e8),
                dict(K=c8.bfloat16(), V=c8.bfloat16(), K_exp=e8, V_exp=e8)):
        with pytest.raises(ValueError):
            wk.wk_cache_attention_workspace(bad, q, 1, 6, 9)
