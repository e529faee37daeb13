"""Calls of the sequence kernels at the edges of what the header allows: maxima of zero, caches without pages."""
import pytest
import torch

import recsys_feature_interaction_b200 as wk
from tests import seq_util as U
from tests.test_gpu_seq import DT, Cached, Jagged, _attend, _ok, _rand, _status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from recsys_feature_interaction_b200 import build
    build.build()
    wk.lib()


@pytest.mark.parametrize("bits", [8, 16])
def test_a_maximum_of_zero_is_told(bits):
    """Sequences longer than a maximum of 0 set the status word, as those longer than any other; batches whose
    sequences are all empty have nothing to write."""
    gen = torch.Generator().manual_seed(1)
    j = Jagged([3, 2], [700, 40], 2, 2, 64, "bf16")
    c = Cached([100, 60], 2, 64, "bf16", 16, bits)
    q = _rand(gen, c.dt, 2, 4, 64)
    k = _rand(gen, c.dt, 4, 2, 64)
    K, V = (torch.full((170, 2, 64), 7.0, dtype=c.dt, device="cuda") for _ in range(2))
    held = {name: t.view(torch.uint8).clone() for name, t in c.cache.items()}

    def calls(off, q_off, new_off, out_off):
        j.max_q, j.q_off = 0, off
        O, L = j.forward()
        yield O, L
        yield _attend(c, q, q_off, 0, True)
        wk.wk_cache_write(c.cache, k, k, new_off, c.table, c.lens, 0)
        for name in held:
            assert torch.equal(held[name], c.cache[name].view(torch.uint8))
        yield ()
        wk.wk_cache_read(c.cache, c.table, c.lens, out_off, K, V, 0)
        yield K, V

    for out in calls(U.offsets([3, 2]), U.offsets([1, 1]), U.offsets([3, 1]), U.offsets([100, 60])):
        assert _status() == wk.WK_ERR_DEVICE
        for t in out:
            assert (t == 7.0).all()
    none = U.offsets([0, 0])
    c.lens.zero_()
    for out in calls(none, none, none, none):
        _ok()
        for t in out:
            assert (t == 7.0).all()
    # a step with fewer bytes of workspace than the smallest of a longer one
    assert wk.wk_xattn_workspace(j.q, j.k, 2, 0, 700) == 0


@pytest.mark.parametrize("n", [1, 70])
@pytest.mark.parametrize("bits,dt", [(8, "bf16"), (8, "f16"), (16, "bf16"), (16, "f16")])
@pytest.mark.parametrize("pages,width", [(0, 0), (0, 3), (4, 0)])
@pytest.mark.parametrize("causal", [True, False])
def test_a_cache_that_holds_nothing_yet(causal, pages, width, bits, dt, n):
    """Empty histories over no pages, or a table without columns: zeros, as over no keys at all. A history that is
    not empty has no place there, and is told."""
    gen = torch.Generator().manual_seed(2)
    kind = torch.float8_e4m3fn if bits == 8 else DT[dt]
    cache = {x: torch.zeros(pages, 2, 16, 64, dtype=torch.uint8 if bits == 8 else kind, device="cuda").view(kind)
             for x in ("K", "V")}
    if bits == 8:
        cache.update({x: torch.zeros(pages, 2, 16, dtype=torch.uint8, device="cuda") for x in ("K_exp", "V_exp")})
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = _rand(gen, DT[dt], n + 1, 4, 64)
    off = U.offsets([n, 1])
    for most, keys in ((0, 0), (900, 0), (900, 5)):
        O, lse = torch.full_like(q, 7.0), torch.full((n + 1, 4), 7.0, device="cuda")
        need = wk.wk_cache_attention_workspace(cache, q, 2, n, most)
        ws = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
        lens[0] = keys
        wk.wk_cache_attention(cache, q, O, off, table, lens, n, most, causal=causal, lse=lse, workspace=ws)
        if keys:
            assert _status() == wk.WK_ERR_DEVICE
            assert (O[n:] == 0).all()
        else:
            _ok()
            assert (O == 0).all() and torch.isneginf(lse).all()
        K, V = (torch.full((7, 2, 64), 7.0, dtype=DT[dt], device="cuda") for _ in range(2))
        wk.wk_cache_read(cache, table, lens, U.offsets([5, 2]), K, V, most)
        if keys:
            assert _status() == wk.WK_ERR_DEVICE
        else:
            _ok()
        assert (K == 7.0).all() and (V == 7.0).all()


def test_broken_boundaries_of_fp16_gradients():
    """Boundaries past the tensors, decreasing or negative, and maxima that are too small: told, and kept inside."""
    j = Jagged([20, 30], [50, 90], 2, 2, 64, "f16")
    O, L = j.forward()
    good = j.backward(O, L)
    _ok()
    for q_off, kv_off in (([0, 20, 99], [0, 50, 140]), ([0, 20, 50], [0, 50, 200]), ([0, 20, 50], [0, 50, 10]),
                          ([-7, 20, 50], [0, 50, 140]), ([0, 20, 50], [2000000000, -5, 140])):
        j.q_off, j.kv_off = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (q_off, kv_off))
        j.backward(O, L)
        assert _status() == wk.WK_ERR_DEVICE
    j.q_off, j.kv_off = U.offsets([20, 30]), U.offsets([50, 90])
    for most in ((29, 90), (30, 89), (0, 90), (30, 0)):
        j.max_q, j.max_kv = most
        j.backward(O, L)
        assert _status() == wk.WK_ERR_DEVICE
    j.max_q, j.max_kv = 30, 90
    again = j.backward(O, L)
    _ok()
    for a, b in zip(good, again):
        assert torch.equal(a[:50], b[:50])
