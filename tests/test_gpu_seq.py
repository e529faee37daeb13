"""Attention over behaviour sequences on the GPU against the fp64 formulas: the jagged cross
attention, its gradients, the paged cache and attention over it. Error bounds are derived in
tests/seq_util.py from where the kernels round; nothing is compared by a chosen tolerance.
"""
import numpy as np
import pytest
import torch

import oracle
import recsys_feature_interaction_b200 as wk
from tests import seq_util as U

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from recsys_feature_interaction_b200 import build
    build.build()
    wk.lib()


def _ok():
    torch.cuda.synchronize()
    assert wk.wk_device_status() == wk.WK_OK


def _rand(gen, dt, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen) * std).to(dt).cuda()


class Jagged:
    """Inputs of a jagged batch with `behind` rows of NaN after the last sequence."""

    def __init__(self, n, kv, hq, hk, d, dt, std=1.0, seed=0, behind=3):
        gen = torch.Generator().manual_seed(seed)
        self.n, self.kv, self.hq, self.hk, self.d, self.dt = n, kv, hq, hk, d, DT[dt]
        self.q = _rand(gen, self.dt, sum(n) + behind, hq, d, std=std)
        self.k = _rand(gen, self.dt, sum(kv) + behind, hk, d)
        self.v = _rand(gen, self.dt, sum(kv) + behind, hk, d)
        self.g = _rand(gen, self.dt, sum(n) + behind, hq, d)
        for t, m in ((self.q, sum(n)), (self.k, sum(kv)), (self.v, sum(kv)), (self.g, sum(n))):
            t[m:] = float("nan")
        self.q_off, self.kv_off = U.offsets(n), U.offsets(kv)
        self.max_q, self.max_kv = max(n), max(kv)

    def workspace(self, backward):
        need = wk.wk_xattn_workspace(self.q, self.k, len(self.n), self.max_q, self.max_kv, backward=backward)
        return torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")

    def forward(self, scale=0.0, lens=None, ws=None, lse=True):
        O = torch.full_like(self.q, 7.0)
        L = torch.full(self.q.shape[:2], 7.0, device="cuda") if lse else None
        wk.wk_xattn_forward(self.q, self.k, self.v, O, self.q_off, self.kv_off, self.max_q, self.max_kv, kv_lens=lens,
                            lse=L, scale=scale, workspace=self.workspace(False) if ws is None else ws)
        return O, L

    def backward(self, O, L, scale=0.0, lens=None):
        grads = [torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda") for t in (self.q, self.k, self.v)]
        wk.wk_xattn_backward(self.q, self.k, self.v, O, L, self.g, *grads, self.q_off, self.kv_off, self.max_q,
                             self.max_kv, kv_lens=lens, scale=scale, workspace=self.workspace(True))
        return grads

    def check(self, O, L=None, grads=None, scale=0.0, lens=None):
        """Every sequence against its bounds, and that no row behind the last one was written."""
        scale = scale or 1.0 / np.sqrt(self.d)
        qa = ka = 0
        q, k, v, g = (U.f64(t) for t in (self.q, self.k, self.v, self.g))
        got = {"O": U.f64(O)}
        if L is not None:
            got["lse"] = U.f64(L)
        if grads is not None:
            got.update(zip(("dQ", "dK", "dV"), (U.f64(t) for t in grads)))
        for b, (n, kv) in enumerate(zip(self.n, self.kv)):
            use = kv if lens is None else lens[b]
            want = U.bounds(q[qa:qa + n], k[ka:ka + use], v[ka:ka + use], self.dt, scale, [use] * n,
                            g[qa:qa + n] if grads is not None else None)
            for name in got:
                at, m = (qa, n) if name in ("O", "lse", "dQ") else (ka, use)
                U.check("%s of sequence %d" % (name, b), got[name][at:at + m], *want[name])
                if name in ("dK", "dV"):
                    assert (got[name][ka + use:ka + kv] == 0).all(), "padding rows of %s" % name
            qa, ka = qa + n, ka + kv
        for name, t in got.items():
            assert (t[qa if name in ("O", "lse", "dQ") else ka:] == 7.0).all(), "%s behind the last sequence" % name


SHAPES = [
    # n, kv, q heads, kv heads, d, std of q
    ([1], [1], 1, 1, 64, 1.0),
    ([1, 1, 1], [250, 1, 63], 4, 4, 64, 1.0),
    ([3, 0, 5, 2], [0, 10, 129, 128], 2, 1, 32, 1.0),
    ([64, 64], [2048, 0], 4, 2, 128, 1.0),
    ([130, 1, 77], [300, 513, 64], 6, 2, 128, 4.0),
    ([200], [1000], 1, 1, 160, 6.0),
    ([17, 129], [65, 640], 5, 1, 160, 1.0),
    ([9] * 40, list(range(40)), 3, 3, 32, 2.0),
    ([512], [700], 2, 2, 64, 3.0),
    ([2], [9000], 8, 2, 128, 1.0),
    ([1] * 5, [4097, 0, 3, 1500, 64], 10, 2, 160, 1.0),
    ([3, 5], [700, 130], 64, 1, 32, 1.0),    # 64 query heads share a key head: two tokens to a tile
    ([7, 2], [600, 31], 48, 1, 64, 1.0),
    ([2, 40], [900, 129], 22, 2, 128, 1.0),  # 11 to a key head: tiles of 121 rows, blocks of 55
    ([0, 0, 4], [10, 600, 0], 2, 2, 64, 1.0),
]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n,kv,hq,hk,d,std", SHAPES)
def test_forward(n, kv, hq, hk, d, std, dt):
    j = Jagged(n, kv, hq, hk, d, dt, std)
    O, L = j.forward()
    _ok()
    j.check(O, L)
    O2, _ = j.forward(lse=False)
    _ok()
    assert torch.equal(O.view(torch.int16), O2.view(torch.int16))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n,kv,hq,hk,d,std", SHAPES)
def test_backward(n, kv, hq, hk, d, std, dt):
    j = Jagged(n, kv, hq, hk, d, dt, std)
    O, L = j.forward()
    grads = j.backward(O, L)
    _ok()
    j.check(O, L, grads)
    again = j.backward(O, L)
    _ok()
    for a, b in zip(grads, again):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)), "two calls differ"


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("d", [32, 64, 128, 160])
def test_padded_batch_with_poisoned_padding(d, dt):
    """kv_lens below the room of a sequence; the padding and the neighbours hold NaN and infinities."""
    lens = [0, 1, 70, 128, 191]
    j = Jagged([5, 33, 1, 65, 128], [192] * 5, 4, 2, d, dt)
    for b, l in enumerate(lens):
        j.k[b * 192 + l:(b + 1) * 192] = float("nan")
        j.v[b * 192 + l:(b + 1) * 192] = float("inf")
    t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    O, L = j.forward(lens=t)
    grads = j.backward(O, L, lens=t)
    _ok()
    j.check(O, L, grads, lens=lens)


def test_much_padding():
    """Far more padding than keys, an odd number of rows of it."""
    lens = [3, 0, 1500]
    j = Jagged([4, 2, 3], [1537, 4099, 1500], 2, 2, 160, "bf16")
    t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    O, L = j.forward(lens=t)
    grads = j.backward(O, L, lens=t)
    _ok()
    j.check(O, L, grads, lens=lens)


@pytest.mark.parametrize("d", [64, 160])
def test_a_poisoned_neighbour_stays_its_own(d):
    """Sequence 1 of three holds NaN in q, k, v and dO: the others' results do not change."""
    j = Jagged([70, 10, 65], [100, 37, 213], 2, 2, d, "bf16")
    clean = j.forward()
    cg = j.backward(*clean)
    for t, off in ((j.q, j.q_off), (j.k, j.kv_off), (j.v, j.kv_off), (j.g, j.q_off)):
        t[off[1]:off[2]] = float("nan")
    O, L = j.forward()
    grads = j.backward(O, L)
    _ok()
    for a, b, off in ((clean[0], O, j.q_off), (cg[0], grads[0], j.q_off), (cg[1], grads[1], j.kv_off),
                      (cg[2], grads[2], j.kv_off)):
        for lo, hi in ((off[0], off[1]), (off[2], off[3])):
            assert torch.equal(a[lo:hi], b[lo:hi])
    assert torch.isnan(O[j.q_off[1]:j.q_off[2]].float()).all()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_strided_tokens_and_shared_keys(dt):
    """Q, K, V as slices of one fused projection, an explicit scale, and V = K."""
    gen = torch.Generator().manual_seed(3)
    n, kv, hq, hk, d = [40, 3], [40, 3], 4, 2, 64
    fused = _rand(gen, DT[dt], 43, hq + 2 * hk, d)
    j = Jagged(n, kv, hq, hk, d, dt, behind=0)
    j.q, j.k, j.v = fused[:, :hq], fused[:, hq:hq + hk], fused[:, hq + hk:]
    O, L = (torch.empty(43, hq, d, dtype=DT[dt], device="cuda"), torch.empty(43, hq, device="cuda"))
    wk.wk_xattn_forward(j.q, j.k, j.v, O, j.q_off, j.kv_off, 40, 40, lse=L, scale=0.3, workspace=j.workspace(False))
    grads = [torch.empty(43, h, d, dtype=DT[dt], device="cuda") for h in (hq, hk, hk)]
    wk.wk_xattn_backward(j.q, j.k, j.v, O, L, j.g, *grads, j.q_off, j.kv_off, 40, 40, scale=0.3,
                         workspace=j.workspace(True))
    _ok()
    j.check(O, L, grads, scale=0.3)
    j.v = j.k
    O, L = j.forward()
    _ok()
    j.check(O, L)


def test_scores_of_extreme_size():
    """Rows whose scores reach thousands, equal scores, and one key that outweighs all others."""
    j = Jagged([4], [300], 1, 1, 64, "bf16", behind=0)
    j.q[0] = 100.0
    j.k[:, 0] = (j.k[:, 0] * 4).round() / 4
    j.q[1] = 0.0
    j.k[211] = 3.0
    j.q[2] = 50.0
    O, L = j.forward()
    _ok()
    j.check(O, L)


def test_gradients_against_differences():
    """Directional differences of the fp64 forward agree with the kernel's gradients within their bounds."""
    j = Jagged([6, 9], [20, 11], 2, 1, 32, "f16", behind=0)
    O, L = j.forward()
    grads = j.backward(O, L)
    _ok()
    gen = np.random.RandomState(0)
    ten = [U.f64(t) for t in (j.q, j.k, j.v)]
    dO = U.f64(j.g)

    def loss(q, k, v):
        s = 0.0
        qa = ka = 0
        for n, kv in zip(j.n, j.kv):
            s += (oracle.sequence_attention(q[qa:qa + n], k[ka:ka + kv], v[ka:ka + kv])[0] * dO[qa:qa + n]).sum()
            qa, ka = qa + n, ka + kv
        return s

    for i in range(3):
        r = gen.randn(*ten[i].shape)
        h = 1e-5
        args = [list(ten), list(ten)]
        args[0][i], args[1][i] = ten[i] + h * r, ten[i] - h * r
        want = (loss(*args[0]) - loss(*args[1])) / (2 * h)
        qa = ka = 0
        bound = 0.0
        for n, kv in zip(j.n, j.kv):
            w = U.bounds(ten[0][qa:qa + n], ten[1][ka:ka + kv], ten[2][ka:ka + kv], torch.float16, 1 / np.sqrt(32),
                         [kv] * n, dO[qa:qa + n])[("dQ", "dK", "dV")[i]][1]
            lo = qa if i == 0 else ka
            bound += (w * np.abs(r[lo:lo + w.shape[0]])).sum()
            qa, ka = qa + n, ka + kv
        assert abs((U.f64(grads[i]) * r).sum() - want) <= bound + 1e-6 * abs(want)


# ------------------------------------------------------------------------ the paged cache

class Cached:
    """A cache of random pages, a table that scatters the sequences over them."""

    def __init__(self, kv, hk, d, dt, page, bits, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.kv, self.hk, self.d, self.dt, self.page = kv, hk, d, DT[dt], page
        each = [-(-x // page) for x in kv]
        pages = sum(each) + 3
        ids = torch.randperm(pages, generator=gen, dtype=torch.int64).to(torch.int32)
        width = max(1, max(each))
        table = torch.full((len(kv), width), -1, dtype=torch.int32)  # entries past the end name no page
        at = 0
        for i, e in enumerate(each):
            table[i, :e] = ids[at:at + e]
            at += e
        self.table, self.lens = table.cuda(), torch.tensor(kv, dtype=torch.int32, device="cuda")
        self.host_table = table.numpy()
        shape = (pages, hk, page, d)
        if bits == 8:
            self.cache = {"K": torch.randint(0, 127, shape, generator=gen).to(torch.uint8).cuda(),
                          "V": torch.randint(0, 127, shape, generator=gen).to(torch.uint8).cuda(),
                          "K_exp": torch.randint(117, 122, shape[:3], generator=gen).to(torch.uint8).cuda(),
                          "V_exp": torch.randint(110, 130, shape[:3], generator=gen).to(torch.uint8).cuda()}
            for name in ("K", "V"):  # both signs
                sign = torch.randint(0, 2, shape, generator=gen).to(torch.uint8).cuda() * 128
                self.cache[name] = (self.cache[name] + sign).view(torch.float8_e4m3fn)
        else:
            self.cache = {"K": _rand(gen, self.dt, *shape), "V": _rand(gen, self.dt, *shape)}

    def values(self, name):
        x = self.cache[name].float().double().cpu().numpy()
        if self.cache.get("K_exp") is not None:
            e = self.cache[name + "_exp"].cpu().numpy().astype(np.int64)
            x = np.where((e == 255)[..., None], np.nan, x * np.ldexp(1.0, e - 127)[..., None])
        return x

    def sequence(self, held, b):
        """[len, hk, d] of sequence b out of values()."""
        pos = np.arange(self.kv[b])
        return held[self.host_table[b][pos // self.page], :, pos % self.page]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("d", [32, 64, 128, 160])
def test_write_quantises_as_defined(d, page, dt):
    """New tokens into an 8-bit cache: the exact values and exponents, nothing else touched, and back again."""
    gen = torch.Generator().manual_seed(d + page)
    n, kv, hk = [1, 0, 37, 130, 5], [1, 50, 37, 300, 129], 3
    c = Cached(kv, hk, d, dt, page, 8)
    before = {k: v.view(torch.uint8).clone() for k, v in c.cache.items()}
    tokens = sum(n)
    k = _rand(gen, c.dt, tokens + 2, hk, d)
    v = _rand(gen, c.dt, tokens + 2, hk, d, std=30.0)
    k *= torch.exp2(torch.randint(-14, 6, (tokens + 2, hk, 1), generator=gen).float()).to(c.dt).cuda()
    k[0, 0] = 0.0                      # a row of zeros
    v[1, 1] = 0.0
    v[1, 1, 3] = 448.0                 # at the border of an exponent
    v[2, 0] = 0.0
    v[2, 0, d - 1] = 450.0
    k[3, 2, 5] = float("inf")
    v[4, 0, 0] = float("nan")
    wk.wk_cache_write(c.cache, k, v, U.offsets(n), c.table, c.lens, max(n))
    _ok()
    expect = {key: t.cpu().numpy().copy() for key, t in before.items()}
    for name, src in (("K", k), ("V", v)):
        vals, exps = oracle.cache_quantise(U.f64(src))
        got_v = U.f64(c.cache[name].float())
        at = 0
        for b in range(len(n)):
            for i in range(n[b]):
                pos = kv[b] - n[b] + i
                pg, r = c.host_table[b][pos // page], pos % page
                ge = c.cache[name + "_exp"][pg, :, r].cpu().numpy()
                assert np.array_equal(ge, exps[at + i]), (name, b, i)
                fin = ge != 255
                assert np.array_equal(got_v[pg, :, r][fin], vals[at + i][fin]), (name, b, i)
                expect[name][pg, :, r] = c.cache[name].view(torch.uint8)[pg, :, r].cpu().numpy()
                expect[name + "_exp"][pg, :, r] = ge
            at += n[b]
    for key in expect:
        assert np.array_equal(expect[key], c.cache[key].view(torch.uint8).cpu().numpy()), "%s: other rows changed" % key


@pytest.mark.parametrize("dt,bits", [("bf16", 8), ("f16", 8), ("bf16", 16), ("f16", 16)])
@pytest.mark.parametrize("page,d", [(16, 160), (32, 32), (64, 128), (128, 64)])
def test_read_back(page, d, dt, bits):
    kv = [0, 1, 77, page, 3 * page + 1]
    c = Cached(kv, 2, d, dt, page, bits)
    if bits == 8:
        c.cache["K_exp"][int(c.host_table[2][0]), 1, 2] = 255
    K, V = (torch.full((sum(kv) + 4, 2, d), 7.0, dtype=c.dt, device="cuda") for _ in range(2))
    wk.wk_cache_read(c.cache, c.table, c.lens, U.offsets(kv), K, V, max(kv))
    _ok()
    for name, got in (("K", K), ("V", V)):
        held = c.values(name)
        want = np.concatenate([c.sequence(held, b) for b in range(len(kv))])
        want = torch.from_numpy(want).float().to(c.dt)  # exact in fp32; one rounding to the output's type
        assert torch.equal(torch.nan_to_num(got[:sum(kv)].cpu()), torch.nan_to_num(want))
        assert torch.equal(torch.isnan(got[:sum(kv)].cpu()), torch.isnan(want))
        assert (got[sum(kv):] == 7.0).all()


def test_write_to_16_bits_and_strides():
    gen = torch.Generator().manual_seed(5)
    c = Cached([40, 9], 2, 64, "f16", 16, 16)
    fused = _rand(gen, torch.float16, 21, 7, 64)
    k, v = fused[:, 1:3], fused[:, 4:6]
    wk.wk_cache_write(c.cache, k, v, U.offsets([17, 4]), c.table, c.lens, 17)
    _ok()
    for name, src in (("K", k), ("V", v)):
        held = c.values(name)
        s = U.f64(src)
        assert np.array_equal(c.sequence(held, 0)[23:], s[:17])
        assert np.array_equal(c.sequence(held, 1)[5:], s[17:])


CACHED = [
    # new rows, lengths, q heads, kv heads, d, page
    ([1], [1], 1, 1, 64, 16),
    ([1, 1, 1, 1], [700, 1, 64, 129], 8, 2, 128, 64),
    ([1] * 3, [5000, 31, 2049], 4, 4, 32, 128),
    ([1, 1], [1030, 77], 5, 1, 160, 16),
    ([4, 1, 0, 7], [200, 65, 50, 7], 4, 2, 64, 32),
    ([130, 64], [300, 64], 4, 2, 128, 32),
    ([200], [900], 2, 2, 160, 64),
    ([300, 5], [300, 1200], 8, 1, 64, 16),
    ([129], [129], 3, 3, 32, 128),
    ([2, 1, 3], [700, 300, 3], 4, 1, 128, 64),
    ([3, 2], [1111, 15], 5, 1, 160, 32),
]


def _attend(c, q, q_off, max_q, causal, lse=True):
    O = torch.full_like(q, 7.0)
    L = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    need = wk.wk_cache_attention_workspace(c.cache, q, len(c.kv), max_q, max(c.kv))
    ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    wk.wk_cache_attention(c.cache, q, O, q_off, c.table, c.lens, max_q, max(c.kv), causal=causal, lse=L, workspace=ws)
    return O, L


def _check_attend(c, q, n, O, L, causal):
    held = {x: c.values(x) for x in ("K", "V")}
    at = 0
    for b, m in enumerate(n):
        k, v = c.sequence(held["K"], b), c.sequence(held["V"], b)
        seen = [max(0, c.kv[b] - m + i + 1) if causal else c.kv[b] for i in range(m)]
        want = U.bounds(U.f64(q[at:at + m]), k, v, c.dt, 1 / np.sqrt(c.d), seen)
        U.check("O of sequence %d" % b, U.f64(O[at:at + m]), *want["O"])
        U.check("lse of sequence %d" % b, U.f64(L[at:at + m]), *want["lse"])
        at += m
    assert (O[at:] == 7.0).all() and (L[at:] == 7.0).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dt,bits", [("bf16", 8), ("f16", 8), ("bf16", 16), ("f16", 16)])
@pytest.mark.parametrize("n,kv,hq,hk,d,page", CACHED)
def test_attention_over_the_cache(n, kv, hq, hk, d, page, dt, bits, causal):
    gen = torch.Generator().manual_seed(1)
    c = Cached(kv, hk, d, dt, page, bits)
    q = _rand(gen, c.dt, sum(n) + 2, hq, d, std=0.2 if bits == 8 else 1.0)
    q[sum(n):] = float("nan")
    # rows of the last pages behind the sequences hold NaN
    for b, l in enumerate(kv):
        if l % page:
            p = int(c.host_table[b][l // page])
            if bits == 8:
                c.cache["K_exp"][p, :, l % page:] = 255
                c.cache["V_exp"][p, :, l % page:] = 255
                c.cache["V"].view(torch.uint8)[p, :, l % page:] = 127
            else:
                c.cache["K"][p, :, l % page:] = float("nan")
                c.cache["V"][p, :, l % page:] = float("inf")
    O, L = _attend(c, q, U.offsets(n), max(n), causal)
    _ok()
    _check_attend(c, q, n, O, L, causal)


def test_more_new_tokens_than_positions_leaves_rows_empty():
    """5 query rows of a sequence of 2: the first three see nothing."""
    gen = torch.Generator().manual_seed(1)
    c = Cached([2, 300], 2, 64, "bf16", 16, 8)
    q = _rand(gen, c.dt, 5 + 1, 4, 64, std=0.2)
    O, L = _attend(c, q, U.offsets([5, 1]), 5, True)
    _ok()
    _check_attend(c, q, [5, 1], O, L, True)
    assert (O[:3] == 0).all() and torch.isinf(L[:3]).all()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 70])
@pytest.mark.parametrize("d", [32, 160])
def test_small_values_of_8_bit_rows(d, n, dt):
    """Rows that hold nothing but e4m3's values below its normal range, rows of zeros with the least exponent, and
    exponents far apart."""
    gen = torch.Generator().manual_seed(6)
    c = Cached([300, 40], 1, d, dt, 16, 8)
    for name in ("K", "V"):
        raw = c.cache[name].view(torch.uint8)
        raw[:, :, ::2] = (raw[:, :, ::2] & 0x80) | (raw[:, :, ::2] & 0x07)
        raw[:, :, 5] = 0
        c.cache[name + "_exp"][:, :, 5] = 0
        c.cache[name + "_exp"][:, :, ::2] += 9
    c.cache["V_exp"][:, :, 11] = 100
    q = _rand(gen, c.dt, n + 1, 2, d)
    O, L = _attend(c, q, U.offsets([n, 1]), n, True)
    _ok()
    _check_attend(c, q, [n, 1], O, L, True)


@pytest.mark.parametrize("n", [1, 70])
def test_the_smallest_queries_over_the_largest_keys(n):
    """Queries near the type's smallest normal value, 8-bit keys with exponents to match: ordinary scores."""
    gen = torch.Generator().manual_seed(12)
    c = Cached([300, 40], 1, 64, "bf16", 16, 8)
    c.cache["K_exp"] += 115
    q = _rand(gen, c.dt, n + 1, 2, 64).float() * 2.0 ** -116
    q = torch.where(q.abs() < 2.0 ** -122, 0.0, q).to(c.dt)
    O, L = _attend(c, q, U.offsets([n, 1]), n, True)
    _ok()
    _check_attend(c, q, [n, 1], O, L, True)


@pytest.mark.parametrize("n", [1, 70])
def test_a_row_that_is_not_finite_shows(n):
    """A NaN row that takes part makes the rows that see it NaN, and no others."""
    gen = torch.Generator().manual_seed(1)
    c = Cached([200, 90], 1, 64, "bf16", 16, 8)
    c.cache["K_exp"][int(c.host_table[0][3]), 0, 4] = 255
    q = _rand(gen, c.dt, n + 1, 2, 64, std=0.2)
    O, _ = _attend(c, q, U.offsets([n, 1]), n, False)
    _ok()
    assert torch.isnan(O[:n].float()).all() and torch.isfinite(O[n:].float()).all()


# ------------------------------------------------------------------ a run of them together

@pytest.mark.parametrize("bits,dt", [(8, "bf16"), (16, "f16")])
def test_history_then_steps(bits, dt):
    """A history is written, attended as a prompt, grows by one event per step, is read back and trained on:
    every result against the definition on what the cache holds."""
    gen = torch.Generator().manual_seed(9)
    hq, hk, d, page = 4, 2, 64, 32
    full = [70, 33]
    c = Cached([74, 37], hk, d, dt, page, bits)
    n = list(full)
    for step in range(5):
        new = full if step == 0 else [1, 1]
        c.kv = [f + step for f in full]
        c.lens.copy_(torch.tensor(c.kv, dtype=torch.int32))
        k, v = (_rand(gen, c.dt, sum(new), hk, d) for _ in range(2))
        q = _rand(gen, c.dt, sum(new) + 1, hq, d)
        off = U.offsets(new)
        wk.wk_cache_write(c.cache, k, v, off, c.table, c.lens, max(new))
        O, L = _attend(c, q, off, max(new), True)
        _ok()
        _check_attend(c, q, new, O, L, True)
    kv = c.kv
    j = Jagged([3, 5], kv, hq, hk, d, dt, behind=0)
    wk.wk_cache_read(c.cache, c.table, c.lens, j.kv_off, j.k, j.v, max(kv))
    O, L = j.forward()
    grads = j.backward(O, L)
    _ok()
    j.check(O, L, grads)
    # the candidates' rows over the cache give the rows over what was read, up to the read's rounding
    O2, L2 = _attend(c, j.q, j.q_off, 5, False)
    _ok()
    _check_attend(c, j.q, [3, 5], O2, L2, False)


# ------------------------------------------------------------ streams, graphs, broken tables

def test_captured_on_another_stream_and_replayed():
    """A training step and a cache step, captured, replayed on new values; two graphs with a workspace each,
    replayed side by side, give what the eager calls give."""
    j = Jagged([40, 1], [300, 2500], 4, 2, 64, "bf16")
    O, L = j.forward()
    grads = j.backward(O, L)
    _ok()
    graphs = []
    for _ in range(2):
        ws = [j.workspace(False), j.workspace(True)]
        out = [torch.zeros_like(O), torch.zeros_like(L)] + [torch.zeros_like(t) for t in grads]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            wk.wk_xattn_forward(j.q, j.k, j.v, out[0], j.q_off, j.kv_off, j.max_q, j.max_kv, lse=out[1],
                                workspace=ws[0])
            wk.wk_xattn_backward(j.q, j.k, j.v, out[0], out[1], j.g, *out[2:], j.q_off, j.kv_off, j.max_q, j.max_kv,
                                 workspace=ws[1])
        graphs.append((g, out, ws, torch.cuda.Stream()))
    j.q.copy_(torch.where(torch.isnan(j.q), j.q, -j.q))
    torch.cuda.synchronize()
    for g, _, _, s in graphs * 3:
        with torch.cuda.stream(s):
            g.replay()
    O, L = j.forward()
    grads = j.backward(O, L)
    _ok()
    real = [41, 41, 41, 2800, 2800]
    for _, out, _, _ in graphs:
        for a, b, m in zip(out, [O, L, *grads], real):
            assert torch.equal(a[:m], b[:m])


def test_lengths_change_between_replays():
    """The grid goes by max_q and max_kv; the lengths are read when the graph runs."""
    gen = torch.Generator().manual_seed(2)
    c = Cached([600, 40], 2, 128, "bf16", 64, 8)
    q = _rand(gen, c.dt, 2, 4, 128, std=0.2)
    off = U.offsets([1, 1])
    O, L = torch.empty_like(q), torch.empty(2, 4, device="cuda")
    ws = torch.empty(max(1, wk.wk_cache_attention_workspace(c.cache, q, 2, 1, 600)), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        wk.wk_cache_attention(c.cache, q, O, off, c.table, c.lens, 1, 600, lse=L, workspace=ws)
    for kv in ([600, 40], [1, 39], [333, 0]):
        c.kv = kv
        c.lens.copy_(torch.tensor(kv, dtype=torch.int32))
        g.replay()
        _ok()
        _check_attend(c, q, [1, 1], O, L, False)


def _status():
    torch.cuda.synchronize()
    first, second = wk.wk_device_status(), wk.wk_device_status()
    assert second == wk.WK_OK  # reading it clears it
    return first


def test_broken_tables_are_told_and_kept_inside():
    """Pages that do not exist, lengths past the table, boundaries past the tensors, sequences longer than max_q
    or max_kv: the status word says so, and sequences that are in order keep their results. What the index
    arithmetic answers to these is tested without a GPU in test_seq_cpu.py."""
    gen = torch.Generator().manual_seed(4)
    c = Cached([100, 60], 2, 64, "bf16", 16, 8)
    q = _rand(gen, c.dt, 2, 4, 64, std=0.2)
    off = U.offsets([1, 1])
    good, _ = _attend(c, q, off, 1, False)
    _ok()
    for bad in (-1, 1 << 30, c.cache["K"].shape[0]):
        keep = c.table.clone()
        c.table[0, 2] = bad
        O, _ = _attend(c, q, off, 1, False)
        assert _status() == wk.WK_ERR_DEVICE
        assert torch.equal(O[1], good[1])
        k = _rand(gen, c.dt, 70, 2, 64)
        wk.wk_cache_write(c.cache, k, k, U.offsets([70, 0]), c.table, c.lens, 70)
        assert _status() == wk.WK_ERR_DEVICE
        K, V = (torch.zeros(160, 2, 64, dtype=c.dt, device="cuda") for _ in range(2))
        wk.wk_cache_read(c.cache, c.table, c.lens, U.offsets([100, 60]), K, V, 100)
        assert _status() == wk.WK_ERR_DEVICE
        c.table.copy_(keep)
        good, _ = _attend(c, q, off, 1, False)
        _ok()
    lens = c.lens.clone()
    for bad in (-5, 113, 1 << 30):
        c.lens[0] = bad
        O, _ = _attend(c, q, off, 1, False)
        assert _status() == wk.WK_ERR_DEVICE
        assert torch.equal(O[1], good[1])
    c.lens.copy_(lens)
    j = Jagged([20, 30], [50, 90], 2, 2, 64, "bf16")
    O, L = j.forward()
    _ok()
    for q_off, kv_off in (([0, 20, 99], [0, 50, 140]), ([0, 20, 50], [0, 50, 200]), ([0, 20, 50], [0, 50, 10]),
                          ([-7, 20, 50], [0, 50, 140])):
        j.q_off, j.kv_off = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (q_off, kv_off))
        j.forward()
        assert _status() == wk.WK_ERR_DEVICE
        j.backward(O, L)
        assert _status() == wk.WK_ERR_DEVICE
    j.q_off, j.kv_off = U.offsets([20, 30]), U.offsets([50, 90])
    j.max_kv = 89
    j.forward()
    assert _status() == wk.WK_ERR_DEVICE
    j.max_kv, j.max_q = 90, 29
    j.forward()
    assert _status() == wk.WK_ERR_DEVICE
    j.max_q = 30
    O2, _ = j.forward()
    _ok()
    assert torch.equal(O2[:50], O[:50])


def test_a_flag_left_unread_spoils_nothing():
    """A broken table in one sequence, its status not read: the others of that call, and a later call, are right."""
    gen = torch.Generator().manual_seed(4)
    c = Cached([600, 700], 2, 64, "bf16", 16, 16)
    q = _rand(gen, c.dt, 60, 4, 64)
    off = U.offsets([30, 30])
    good, lse = _attend(c, q, off, 30, True)
    _ok()
    keep = c.table.clone()
    c.table[0, 20] = 1 << 20
    O, _ = _attend(c, q, off, 30, True)
    assert torch.equal(O[30:], good[30:])
    c.table.copy_(keep)
    O, L = _attend(c, q, off, 30, True)
    assert torch.equal(O, good) and torch.equal(L, lse)
    assert _status() == wk.WK_ERR_DEVICE


# ---------------------------------------------------------------- sizes at the edges

@pytest.mark.parametrize("rows", [1, 23])
def test_thousands_of_short_sequences(rows):
    """More units than blocks of the grid by far, most of them of one key block or none."""
    r = np.random.RandomState(5)
    n = [int(x) for x in r.randint(0, rows + 1, 3000)]
    kv = [int(x) for x in r.randint(0, 40, 3000)]
    n[0], kv[1] = rows, 700  # some are cut
    j = Jagged(n, kv, 2, 2, 32, "bf16")
    O, L = j.forward()
    grads = j.backward(O, L)
    _ok()
    j.check(O, L, grads)


@pytest.mark.parametrize("n", [1, 20])
def test_a_long_sequence_among_short_ones(n):
    """One sequence is most of the work: it is cut over nearly every block."""
    gen = torch.Generator().manual_seed(8)
    c = Cached([70001, 5, 300], 1, 64, "bf16", 128, 8)
    q = _rand(gen, c.dt, n + 2, 2, 64, std=0.2)
    O, L = _attend(c, q, U.offsets([n, 1, 1]), n, True)
    _ok()
    _check_attend(c, q, [n, 1, 1], O, L, True)


def test_nothing_at_all():
    """No keys anywhere, no rows anywhere, no sequences: zeros, or nothing written."""
    j = Jagged([5, 0], [0, 0], 2, 2, 64, "bf16", behind=0)
    j.max_kv = 0
    O, L = j.forward()
    grads = j.backward(O, L)
    _ok()
    assert (O == 0).all() and torch.isneginf(L).all() and (grads[0] == 0).all()
    j = Jagged([0, 0], [5, 300], 2, 2, 64, "bf16", behind=0)
    j.max_q = 0
    O, L = j.forward()
    grads = j.backward(O, L)
    _ok()
    assert (grads[1] == 0).all() and (grads[2] == 0).all()
    empty = torch.zeros(1, dtype=torch.int32, device="cuda")
    j.q_off = j.kv_off = empty
    j.n = []
    wk.wk_xattn_forward(j.q, j.k, j.v, O, empty, empty, 0, 0, workspace=j.workspace(False))
    _ok()


@pytest.mark.parametrize("d", [64, 160])
def test_infinities_in_keys_that_take_part(d):
    """An infinite key gives NaN or the winning weight as the definition does; other sequences keep theirs."""
    j = Jagged([40, 40], [200, 200], 1, 1, d, "bf16", behind=0)
    clean, _ = j.forward()
    j.k[5] = float("inf")
    O, _ = j.forward()
    _ok()
    assert torch.isnan(O[:40].float()).all()
    assert torch.equal(O[40:], clean[40:])


def test_two_streams_at_once():
    """Two calls on two streams, each with a workspace of its own, give what they give alone."""
    a = Jagged([64] * 20, [2000] * 20, 4, 2, 128, "bf16", seed=1)
    b = Jagged([3] * 50, [900] * 50, 4, 4, 64, "f16", seed=2)
    alone = []
    for j in (a, b):
        O, L = j.forward()
        alone.append([O, L, *j.backward(O, L)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    keep = [(j.workspace(False), j.workspace(True)) for j in (a, b)]
    outs = []
    torch.cuda.synchronize()
    for j, s, (w0, w1) in zip((a, b), streams, keep):
        with torch.cuda.stream(s):
            O, L = torch.empty_like(j.q), torch.empty(j.q.shape[:2], device="cuda")
            grads = [torch.empty_like(t) for t in (j.q, j.k, j.v)]
            for _ in range(3):
                wk.wk_xattn_forward(j.q, j.k, j.v, O, j.q_off, j.kv_off, j.max_q, j.max_kv, lse=L, workspace=w0)
                wk.wk_xattn_backward(j.q, j.k, j.v, O, L, j.g, *grads, j.q_off, j.kv_off, j.max_q, j.max_kv,
                                     workspace=w1)
            outs.append([O, L, *grads])
    _ok()
    for j, x, y in zip((a, b), outs, alone):
        ends = [sum(j.n)] * 3 + [sum(j.kv)] * 2
        for t, u, m in zip(x, y, ends):
            assert torch.equal(t[:m], u[:m])


def test_a_stream_that_is_not_the_current_one():
    j = Jagged([33, 2], [500, 700], 2, 1, 64, "f16", behind=0)
    want, _ = j.forward()
    _ok()
    s = torch.cuda.Stream()
    O = torch.zeros_like(want)
    ws = j.workspace(False)
    torch.cuda.synchronize()
    wk.wk_xattn_forward(j.q, j.k, j.v, O, j.q_off, j.kv_off, j.max_q, j.max_kv, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(O, want)
