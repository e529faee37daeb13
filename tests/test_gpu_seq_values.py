"""Attention over behaviour sequences on the GPU where the values are far apart, tiny, huge, zero or not finite:
8-bit rows with powers of two of every size, NaN bytes, single infinite scores, fp16 gradients of small and of large
losses.

Bounds, with u half a step of the 16-bit type and e_j = ES + 2^-23 d sum |q k_j| scale of each score (seq_util):
  8-bit caches  key j's weight is off by P_j (u + 2 e_j), and every weight by the row sum's sum_j P_j e_j. Weights
                are held in 16 bits together with their V row's power of two, relative to the row's largest such
                product, so fp16's smallest step adds 2^-25 max_k(P_k 2^x_k) sum_j |v_j| (x the exponents, v
                the e4m3 values).
  fp16 grads    P (dP - delta) enters relative to a power of two at least 2^10 / (|dO| |V|), |dO| the norm of the
                row (dQ) or the largest of the rows that share a key head (dK), |V| the largest of the sequence:
                fp16's smallest step adds 2^-25 2^-10 |dO| |V|. P enters dV times 2^12: 2^-37.
"""
import numpy as np
import pytest
import torch

import recsys_feature_interaction_b200 as wk
from tests import seq_util as U
from tests.test_gpu_seq import Cached, Jagged, _attend, _check_attend, _ok, _rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    from recsys_feature_interaction_b200 import build
    build.build()
    wk.lib()


# ------------------------------------------------------------------ 8-bit rows of every size

def _held(c):
    """{name: (e4m3 values, powers of two)} of the whole cache in float64."""
    return {name: (U.f64(c.cache[name].float()),
                   np.ldexp(1.0, c.cache[name + "_exp"].cpu().numpy().astype(int) - 127)) for name in ("K", "V")}


def _set(c, b, pos, name, values=None, exp=None):
    """Rows `pos` of sequence b: e4m3 values (a number) and / or exponent bytes."""
    pos = np.atleast_1d(pos)
    page = torch.from_numpy(c.host_table[b][pos // c.page].astype(np.int64)).cuda()
    row = torch.from_numpy(pos % c.page).cuda()
    if values is not None:
        x = torch.as_tensor(values, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
        c.cache[name].view(torch.uint8)[page, :, row] = x
    if exp is not None:
        c.cache[name + "_exp"][page, :, row] = torch.as_tensor(exp, dtype=torch.uint8).cuda()


def _check8(c, q, n, O, causal):
    at, held = 0, _held(c)
    u, d = U.half_step(c.dt), c.d
    least = torch.finfo(c.dt).smallest_normal * torch.finfo(c.dt).eps
    for b, m in enumerate(n):
        if m == 0 or c.kv[b] == 0:
            assert (O[at:at + m] == 0).all()
            at += m
            continue
        pos = np.arange(c.kv[b])
        page, row = c.host_table[b][pos // c.page], pos % c.page
        x, (kp, vp) = ([U.expand(held[name][i][page, :, row], q.shape[1]) for name in ("K", "V")] for i in (0, 1))
        k, v = x[0] * kp[..., None], x[1] * vp[..., None]
        qq = U.f64(q[at:at + m])
        seen = np.array([max(0, c.kv[b] - m + i + 1) if causal else c.kv[b] for i in range(m)])
        mask = (np.arange(c.kv[b])[None] < seen[:, None])[:, None]
        S = np.where(mask, np.einsum("nhd,lhd->nhl", qq, k) / np.sqrt(d), -np.inf)
        e = U.ES + 2.0 ** -23 * d * np.einsum("nhd,lhd->nhl", np.abs(qq), np.abs(k)) / np.sqrt(d)
        top = S.max(axis=2, keepdims=True)
        P = np.where(mask, np.exp(S - np.where(np.isfinite(top), top, 0.0)), 0.0)
        P /= np.maximum(P.sum(axis=2, keepdims=True), 1e-300)
        O_ref = np.einsum("nhl,lhd->nhd", P, v)
        A = np.einsum("nhl,lhd->nhd", P, np.abs(v))
        bound = np.einsum("nhl,lhd->nhd", P * (u + 2 * e), np.abs(v)) + 2 * (P * e).sum(axis=2, keepdims=True) * A
        largest = (P * vp.T[None]).max(axis=2, keepdims=True)
        bound += 2.0 ** -25 * largest * np.einsum("nhl,lhd->nhd", np.broadcast_to(mask, P.shape).astype(float),
                                                  np.abs(x[1]))
        U.check("O of sequence %d" % b, U.f64(O[at:at + m]), O_ref, 1.05 * bound + u * np.abs(O_ref) + least)
        at += m


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [1, 3, 70])
@pytest.mark.parametrize("d", [32, 128, 160])
def test_keys_of_zeros(d, n, causal, dt):
    """A history of zero rows (written with exponent 0): the output is the mean of V."""
    gen = torch.Generator().manual_seed(1)
    c = Cached([300, 77], 2, d, dt, 16, 8)
    for b in range(2):
        _set(c, b, np.arange(c.kv[b]), "K", 0.0, 0)
    q = _rand(gen, c.dt, 2 * n, 4, d)
    O, L = _attend(c, q, U.offsets([n, n]), n, causal)
    _ok()
    _check_attend(c, q, [n, n], O, L, causal)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [3, 40])
def test_a_tail_of_zero_keys_in_a_cut_sequence(n, causal, dt):
    """The last blocks' share of a long history holds nothing but zero rows, and ends inside a block of keys."""
    gen = torch.Generator().manual_seed(2)
    c = Cached([40017], 1, 64, dt, 128, 8)
    _set(c, 0, np.arange(30000, 40017), "K", 0.0, 0)
    q = _rand(gen, c.dt, n, 2, 64, std=0.2)
    O, L = _attend(c, q, U.offsets([n]), n, causal)
    _ok()
    _check_attend(c, q, [n], O, L, causal)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n", [2, 70])
@pytest.mark.parametrize("gap", [25, 40, 90])
def test_a_large_value_row_that_the_mask_hides(gap, n, dt):
    """The newest token's V row is 2^gap above all others: only the last row sees it, the others' results are those
    of the small rows. Its key's score is far below, so the last row's are theirs too."""
    gen = torch.Generator().manual_seed(3)
    c = Cached([200, 150], 1, 64, dt, 16, 8)
    c.cache["V_exp"][:] = 118
    for b in range(2):
        _set(c, b, c.kv[b] - 1, "V", exp=118 + gap)
        _set(c, b, c.kv[b] - 1, "K", -1.0, 127 + 9)  # about -700
    q = _rand(gen, c.dt, 2 * n, 2, 64, std=0.2).abs() + 0.01
    O, _ = _attend(c, q, U.offsets([n, n]), n, True)
    _ok()
    _check8(c, q, [n, n], O, True)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 70])
@pytest.mark.parametrize("place", [0, 64, 199])
def test_a_large_value_row_with_next_to_no_weight(place, n, dt):
    """Key `place` has a V row 2^30 above the others' and a score that leaves it a weight of about 2^-46."""
    gen = torch.Generator().manual_seed(4)
    c = Cached([200], 2, 128, dt, 32, 8)
    c.cache["V_exp"][:] = 119
    _set(c, 0, np.arange(200), "K", exp=112)
    _set(c, 0, place, "V", exp=149)
    _set(c, 0, place, "K", -2.0, 127)
    q = torch.full((n, 4, 128), 1.4140625, dtype=c.dt, device="cuda")  # s = -32 for that key
    O, _ = _attend(c, q, U.offsets([n]), n, False)
    _ok()
    _check8(c, q, [n], O, False)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 70])
def test_large_keys_beside_small_ones(n, dt):
    """Keys with exponents 60 above the others' and scores far below: the small ones share the weight by their scores."""
    gen = torch.Generator().manual_seed(5)
    c = Cached([300, 100], 1, 64, dt, 16, 8)
    c.cache["K_exp"][:] = 122
    for b in range(2):
        _set(c, b, np.arange(7, c.kv[b], 50), "K", -1.0, 182)
    q = _rand(gen, c.dt, 2 * n, 2, 64, std=0.1).abs() + 0.01
    O, _ = _attend(c, q, U.offsets([n, n]), n, True)
    _ok()
    _check8(c, q, [n, n], O, True)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n,kv,d,page", [([1, 1], [900, 31], 128, 64), ([4, 2], [100, 3000], 64, 16),
                                         ([80, 33], [700, 33], 160, 32), ([200], [5000], 32, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_value_rows_of_every_size(causal, n, kv, d, page, dt):
    """V's exponents drawn from 60 powers of two below 1, scores that differ."""
    gen = torch.Generator().manual_seed(6)
    c = Cached(kv, 2, d, dt, page, 8)
    c.cache["V_exp"][:] = torch.randint(60, 120, c.cache["V_exp"].shape, generator=gen).to(torch.uint8).cuda()
    q = _rand(gen, c.dt, sum(n), 6, d, std=1.0)
    O, _ = _attend(c, q, U.offsets(n), max(n), causal)
    _ok()
    _check8(c, q, n, O, causal)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("rows,d", [(2, 64), (20, 64), (20, 160)])
def test_hundreds_of_cached_sequences(rows, d, dt):
    """More units than blocks of the grid, of no key to several blocks of keys, rows of every size."""
    gen = torch.Generator().manual_seed(8)
    r = np.random.RandomState(8)
    n = [int(x) for x in r.randint(0, rows + 1, 400)]
    kv = [int(x) for x in np.maximum(r.choice([0, 20, 130, 700], 400) - r.randint(0, 20, 400), 0)]
    c = Cached(kv, 2, d, dt, 16, 8)
    c.cache["V_exp"][:] = torch.randint(80, 124, c.cache["V_exp"].shape, generator=gen).to(torch.uint8).cuda()
    q = _rand(gen, c.dt, sum(n), 4, d, std=0.5)
    O, _ = _attend(c, q, U.offsets(n), rows, True)
    _ok()
    _check8(c, q, n, O, True)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 70])
@pytest.mark.parametrize("byte", [0x7F, 0xFF])
def test_a_nan_byte_in_an_ordinary_row(byte, n, dt):
    """e4m3's NaN in a row with an ordinary exponent: in V one column of the output, in K every row that sees it."""
    gen = torch.Generator().manual_seed(7)
    c = Cached([200, 90], 1, 64, dt, 16, 8)
    q = _rand(gen, c.dt, n + 1, 2, 64, std=0.2)
    off = U.offsets([n, 1])
    good, _ = _attend(c, q, off, n, False)
    _ok()
    page = int(c.host_table[0][3])
    v = c.cache["V"].view(torch.uint8)
    keep = v[page, 0, 4, 37].item()
    v[page, 0, 4, 37] = byte
    O, _ = _attend(c, q, off, n, False)
    _ok()
    assert torch.isnan(O[:n, :, 37].float()).all()
    rest = [i for i in range(64) if i != 37]
    assert torch.equal(O[:, :, rest], good[:, :, rest]) and torch.equal(O[n:], good[n:])
    v[page, 0, 4, 37] = keep
    c.cache["K"].view(torch.uint8)[page, 0, 4, 11] = byte
    O, _ = _attend(c, q, off, n, False)
    _ok()
    assert torch.isnan(O[:n].float()).all() and torch.equal(O[n:], good[n:])


# ------------------------------------------------------------------------ infinite scores

@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 40])
def test_one_infinite_score(n, dt):
    """A single score of +inf makes the softmax NaN, whichever key it belongs to."""
    j = Jagged([n, n], [200, 200], 1, 1, 64, dt, behind=0)
    j.q[:, :, 9] = j.q[:, :, 9].abs() + 0.1
    clean, _ = j.forward()
    for key in [*range(16), 62, 63, 126, 127, 128, 199]:
        keep = j.k[key, 0, 9].item()
        j.k[key, 0, 9] = float("inf")
        O, _ = j.forward()
        _ok()
        assert torch.isnan(O[:n].float()).all(), key
        assert torch.equal(O[n:], clean[n:]), key
        j.k[key, 0, 9] = keep


# ------------------------------------------------------------------------ fp16 gradients

def _grad_bounds(q, k, v, g, scale):
    """{name: (reference, bound)} of one sequence, fp16 (see the head of this file)."""
    n, hq, d = q.shape
    L, hk, _ = k.shape
    u, least = U.half_step(torch.float16), 2.0 ** -24
    ke, ve = U.expand(k, hq), U.expand(v, hq)
    S = np.einsum("nhd,lhd->nhl", q, ke) * scale
    e = (U.ES + 2.0 ** -23 * d * np.einsum("nhd,lhd->nhl", np.abs(q), np.abs(ke)) * scale).max(axis=2, keepdims=True)
    P = np.exp(S - S.max(axis=2, keepdims=True))
    P /= P.sum(axis=2, keepdims=True)
    O = np.einsum("nhl,lhd->nhd", P, ve)
    eO = 1.05 * ((u + 2 * e) * np.einsum("nhl,lhd->nhd", P, np.abs(ve)) + 2.0 ** -25 * np.abs(ve).sum(axis=0)[None])
    G, Gm = np.einsum("nhd,lhd->nhl", g, ve), np.einsum("nhd,lhd->nhl", np.abs(g), np.abs(ve))
    delta = (g * O).sum(axis=2, keepdims=True)
    e_delta = (np.abs(g) * (eO + u * np.abs(O) + least)).sum(axis=2, keepdims=True) \
        + 2.0 ** -23 * d * (np.abs(g) * np.abs(O)).sum(axis=2, keepdims=True)
    dS = P * (G - delta)
    e_dS = (np.abs(dS) * (u + 2 * e) + P * (1 + 2 * e) * (e_delta + 2.0 ** -23 * d * Gm)) * 1.05
    norm = np.sqrt((g ** 2).sum(axis=2, keepdims=True)) * np.sqrt((ve ** 2).sum(axis=2)).max(axis=0)[None, :, None]
    share = np.repeat(norm.max(axis=0).reshape(hk, -1).max(axis=1), hq // hk)[None, :, None]

    def fold(x):
        return x.reshape(L, hk, hq // hk, d).sum(axis=2)

    out = {}
    dQ = np.einsum("nhl,lhd->nhd", dS, ke) * scale
    out["dQ"] = (dQ, np.einsum("nhl,lhd->nhd", e_dS + 2.0 ** -35 * norm, np.abs(ke)) * scale + u * np.abs(dQ) + least)
    dK = fold(np.einsum("nhl,nhd->lhd", dS, q)) * scale
    out["dK"] = (dK, fold(np.einsum("nhl,nhd->lhd", e_dS + 2.0 ** -35 * share, np.abs(q))) * scale + u * np.abs(dK) + least)
    dV = fold(np.einsum("nhl,nhd->lhd", P, g))
    out["dV"] = (dV, fold(np.einsum("nhl,nhd->lhd", P * (u + 2 * e) * 1.05 + 2.0 ** -37, np.abs(g))) + u * np.abs(dV) + least)
    return out


def _check_grads(j, grads, scale, names=("dQ", "dK", "dV")):
    qa = ka = 0
    q, k, v, g = (U.f64(t) for t in (j.q, j.k, j.v, j.g))
    for b, (n, kv) in enumerate(zip(j.n, j.kv)):
        if n and kv:
            want = _grad_bounds(q[qa:qa + n], k[ka:ka + kv], v[ka:ka + kv], g[qa:qa + n], scale)
            for name, t, at, m in zip(("dQ", "dK", "dV"), grads, (qa, ka, ka), (n, kv, kv)):
                if name in names:
                    U.check("%s of sequence %d" % (name, b), U.f64(t[at:at + m]), *want[name])
        qa, ka = qa + n, ka + kv


SMALL = [
    # rows, keys, q heads, kv heads, d
    ([64, 5], [2048, 300], 2, 1, 128),
    ([16], [15000], 2, 1, 64),
    ([40, 300], [130, 4100], 1, 1, 160),
    ([300, 7], [90, 1], 4, 2, 32),
]


@pytest.mark.parametrize("power", [-7, -10, -13])
@pytest.mark.parametrize("n,kv,hq,hk,d", SMALL)
def test_gradients_of_a_small_loss(n, kv, hq, hk, d, power):
    """dO of the size that a mean over a batch gives."""
    j = Jagged(n, kv, hq, hk, d, "f16", behind=0)
    j.g *= 2.0 ** power
    O, L = j.forward()
    grads = j.backward(O, L)
    _ok()
    _check_grads(j, grads, 1 / np.sqrt(d))


def test_weights_below_halfs_normal_range_reach_dv():
    """Keys with softmax weights of 2^-16 to 2^-22: their value gradients are ordinary numbers."""
    j = Jagged([60], [4000], 1, 1, 64, "f16", behind=0)
    j.q[:, :, 0], j.k[:, :, 0] = 1.0, -64.0  # all but the first 8 keys: 13 below
    j.k[:8, :, 0] = 40.0
    j.g *= 64.0
    O, L = j.forward()
    grads = j.backward(O, L)
    _ok()
    _check_grads(j, grads, 1 / 8, ("dV",))


@pytest.mark.parametrize("n,kv,qk,vs,gs", [([2, 3], [4, 100], 2.0 ** -7, 512.0, 4096.0),
                                           ([40], [200], 2.0 ** -6, 1024.0, 8192.0),
                                           ([200, 70], [600, 1000], 2.0 ** -8, 4096.0, 8192.0)])
def test_gradients_of_a_large_loss(n, kv, qk, vs, gs):
    """dO V^T beyond fp16's largest value, gradients within it."""
    j = Jagged(n, kv, 2, 1, 128, "f16", behind=0)
    for t, s in ((j.q, qk), (j.k, qk), (j.v, vs), (j.g, gs)):
        t *= s
    O, L = j.forward()
    grads = j.backward(O, L)
    _ok()
    ref = np.abs(U.f64(j.g)).max() * np.abs(U.f64(j.v)).max()
    assert ref > 65504
    _check_grads(j, grads, 1 / np.sqrt(128))


def test_rows_with_losses_of_different_size():
    """Each row's gradient goes by its own dO; a row without any has none."""
    j = Jagged([50, 20], [1500, 100], 2, 1, 64, "f16", behind=0)
    w = torch.exp2(torch.arange(70, device="cuda") % 13 * -1.0)
    w[::9] = 0.0
    j.g = (j.g.float() * w[:, None, None]).half()
    O, L = j.forward()
    grads = j.backward(O, L)
    _ok()
    _check_grads(j, grads, 1 / 8)
    assert (grads[0][::9] == 0).all()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_a_poisoned_neighbour_of_small_gradients(dt):
    """NaN and infinities in one sequence's values and output gradients leave the others' gradients as they were."""
    j = Jagged([70, 10, 65], [100, 37, 213], 2, 2, 64, dt)
    j.g *= 2.0 ** -10
    clean = j.forward()
    cg = j.backward(*clean)
    for bad in (float("nan"), float("inf")):
        j.v[j.kv_off[1]:j.kv_off[2]] = bad
        j.g[j.q_off[1]:j.q_off[2]] = bad
        grads = j.backward(*j.forward())
        _ok()
        for a, b, off in zip(cg, grads, (j.q_off, j.kv_off, j.kv_off)):
            for lo, hi in ((off[0], off[1]), (off[2], off[3])):
                assert torch.equal(a[lo:hi], b[lo:hi])
