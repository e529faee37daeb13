"""The sequence calls next to the rest of the framework and to one another: a stack's rows over histories into the
WHALE fusion, prompts of thousands of tokens, calls on two branches of one captured graph."""
import numpy as np
import pytest
import torch

import oracle
import recsys_feature_interaction_b200 as wk
from synth import configs as C
from tests import seq_util as U
from tests.gpu_util import f64, max_scaled_err, oracle_weight, to_dev
from tests.test_gpu_seq import Cached, Jagged, _attend, _check_attend, _ok, _rand
from tests.test_gpu_whale import TOL, _ffn_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from recsys_feature_interaction_b200 import build
    build.build()
    wk.lib()


@pytest.mark.parametrize("bits", [0, 8, 16])
def test_stack_rows_over_histories_into_the_fusion(bits):
    """The interaction rows that the 2-layer stack gives attend over their users' histories (jagged, or in a cache,
    one user without any) and enter the module's fusion and FFN."""
    cfg = C.CONFIGS["c2_bf16"]
    batch, n, d, h = 3, cfg["n"], cfg["d"], 256
    layers = [C.make_layer_dev(cfg, l) for l in range(cfg["layers"])]
    stack = wk.wk_stack_create(cfg, layers, max_batch=batch)
    X = C.make_x_dev(cfg, batch)
    Hw = torch.empty_like(X)
    wk.wk_stack_forward(stack, X, Hw)
    torch.cuda.synchronize()
    assert wk.wk_stack_sync_status(stack) == wk.WK_OK
    wk.wk_stack_destroy(stack)

    gen = torch.Generator().manual_seed(1)
    lens = [700, 0, 37]
    K, V = (_rand(gen, torch.bfloat16, sum(lens), 1, d) for _ in range(2))
    Q = Hw.view(batch * n, 1, d)
    q_off, kv_off = U.offsets([n] * batch), U.offsets(lens)
    A = torch.full_like(Q, 7.0)
    if bits == 0:
        ws = torch.empty(max(1, wk.wk_xattn_workspace(Q, K, batch, n, 700)), dtype=torch.uint8, device="cuda")
        wk.wk_xattn_forward(Q, K, V, A, q_off, kv_off, n, 700, workspace=ws)
        k64, v64 = U.f64(K), U.f64(V)
    else:
        c = Cached(lens, 1, d, "bf16", 32, bits)
        wk.wk_cache_write(c.cache, K, V, kv_off, c.table, c.lens, 700)
        A, _ = _attend(c, Q, q_off, n, False)
        held = {x: c.values(x) for x in ("K", "V")}
        k64, v64 = (np.concatenate([c.sequence(held[x], b) for b in range(batch)]) for x in ("K", "V"))
    w = _ffn_weights(d, h, True, "bf16")
    Hf = torch.empty_like(Hw)
    wk.wk_whale_fusion_ffn(Hw, A, {k: to_dev(v) for k, v in w.items()}, Hf, batch * n, d, h, "bf16")
    _ok()
    hw, at = U.f64(Hw), 0
    ow = {k: oracle_weight(v) for k, v in w.items()}
    for b, l in enumerate(lens):
        a, _ = oracle.sequence_attention(hw[b][:, None], k64[at:at + l], v64[at:at + l])
        err = max_scaled_err(f64(Hf[b]), oracle.fusion_ffn(hw[b], a[:, 0], ow))
        assert err <= TOL, (b, err)
        at += l


@pytest.mark.parametrize("dt,bits", [("bf16", 8), ("f16", 8), ("bf16", 16), ("f16", 16)])
@pytest.mark.parametrize("n,kv,hq,hk,d,page", [([2500, 1100], [2500, 3001], 2, 1, 64, 64),
                                               ([1501, 1], [1501, 2000], 5, 1, 160, 16)])
def test_prompts_of_thousands_of_tokens(n, kv, hq, hk, d, page, dt, bits):
    gen = torch.Generator().manual_seed(2)
    c = Cached(kv, hk, d, dt, page, bits)
    q = _rand(gen, c.dt, sum(n) + 2, hq, d, std=0.2 if bits == 8 else 1.0)
    O, L = _attend(c, q, U.offsets(n), max(n), True)
    _ok()
    _check_attend(c, q, n, O, L, True)


@pytest.mark.parametrize("bits,dt", [(8, "f16"), (16, "bf16")])
def test_two_branches_of_one_graph(bits, dt):
    """New tokens are written on one branch while another attends over jagged rows; the step that joins them attends
    over the cache and reads it back. Replayed on new values it gives what the calls give one after another."""
    gen = torch.Generator().manual_seed(3)
    c = Cached([900, 70], 2, 64, dt, 32, bits)
    j = Jagged([40, 3], [600, 90], 4, 2, 64, dt)
    k, v = (_rand(gen, c.dt, 2, 2, 64) for _ in range(2))
    q = _rand(gen, c.dt, 2, 4, 64, std=0.2)
    off, out_off = U.offsets([1, 1]), U.offsets(c.kv)
    ws = [j.workspace(True), torch.empty(max(1, wk.wk_cache_attention_workspace(c.cache, q, 2, 1, 900)),
                                         dtype=torch.uint8, device="cuda")]
    new = lambda: [torch.zeros_like(j.q), torch.zeros(j.q.shape[:2], device="cuda"), torch.zeros_like(q),  # noqa: E731
                   *(torch.zeros(970, 2, 64, dtype=c.dt, device="cuda") for _ in range(2))]

    def step(out, one, two):
        two.wait_stream(one)
        with torch.cuda.stream(two):
            wk.wk_cache_write(c.cache, k, v, off, c.table, c.lens, 1)
        wk.wk_xattn_forward(j.q, j.k, j.v, out[0], j.q_off, j.kv_off, 40, 600, lse=out[1], workspace=ws[0])
        one.wait_stream(two)
        wk.wk_cache_attention(c.cache, q, out[2], off, c.table, c.lens, 1, 900, workspace=ws[1])
        two.wait_stream(one)
        with torch.cuda.stream(two):
            wk.wk_cache_read(c.cache, c.table, c.lens, out_off, out[3], out[4], 900)
        one.wait_stream(two)

    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    got, want = new(), new()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=one):
        step(got, one, two)
    for i in range(3):
        for t in (k, v, q):
            t.copy_(_rand(gen, c.dt, *t.shape, std=0.2))
        j.k[:600] = _rand(gen, c.dt, 600, 2, 64)
        torch.cuda.synchronize()
        graph.replay()
        _ok()
        with torch.cuda.stream(one):
            step(want, one, one)
        _ok()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_a_captured_training_step_on_new_values(dt):
    """A padded training step, captured; replayed with another loss, other lengths and other values, it gives the
    gradients of the eager calls on them."""
    gen = torch.Generator().manual_seed(4)
    j = Jagged([30, 1, 65], [700, 40, 300], 4, 2, 64, dt, behind=0)
    lens = torch.tensor([650, 0, 300], dtype=torch.int32, device="cuda")
    ws = j.workspace(True)
    out = [torch.empty_like(j.q), torch.empty(j.q.shape[:2], device="cuda"),
           *(torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (j.q, j.k, j.v))]

    def step():
        wk.wk_xattn_forward(j.q, j.k, j.v, out[0], j.q_off, j.kv_off, 65, 700, kv_lens=lens, lse=out[1], workspace=ws)
        wk.wk_xattn_backward(j.q, j.k, j.v, out[0], out[1], j.g, *out[2:], j.q_off, j.kv_off, 65, 700, kv_lens=lens,
                             workspace=ws)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for i, (size, use) in enumerate((((1.0), [650, 0, 300]), (2.0 ** -9, [1, 40, 129]), (2.0 ** 5, [700, 0, 0]))):
        lens.copy_(torch.tensor(use, dtype=torch.int32))
        for t in (j.q, j.k, j.v):
            t.copy_(_rand(gen, j.dt, *t.shape))
        j.g.copy_(_rand(gen, j.dt, *j.g.shape, std=size))
        for t in out:
            t.fill_(7.0)
        graph.replay()
        _ok()
        got = [t.clone() for t in out]
        for t in out:
            t.fill_(5.0)
        step()
        _ok()
        for a, b in zip(got, out):
            assert torch.equal(a, b), i
        if size == 1.0 or dt == "bf16":
            j.check(out[0], out[1], out[2:], lens=use)
