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
