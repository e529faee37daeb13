"""Shared by the tests of attention over behaviour sequences: jagged inputs, and for every output
the bound that its error has to stay under, derived from where the kernels round.

With u = eps / 2 of the 16-bit type (half a step, relative) and, per score, e = ES + 2^-23 d
sum |q k| scale (the exponential's error, and fp32 accumulation of d products):
  O    final rounding u |O|; each weight is rounded once (u) and off by e, its share in the row sum
       by e again: (u + 2 e) sum_j P_j |V_j|. Weights below the 16-bit type's smallest step round by
       at most 2^-25 of the largest (fp16): 2^-25 sum_j |V_j|.
  lse  e + 2^-22 |lse|
  dS   = P (dP - delta): P off by 2 e (score, and lse of the forward), delta by sum |dO| (error of the
       stored O), dP by 2^-23 d sum |dO V|; then rounded once (u)
  dQ, dK, dV: sums of |rounded weight error| times |the other operand|, plus the final rounding.
"""
import numpy as np
import torch

ES = 1e-4  # relative error allowed to one exponential (its argument's fp32 rounding included)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def expand(x, hq):
    return np.repeat(x, hq // x.shape[1], axis=1)


def bounds(q, k, v, dtype, scale, seen, dO=None):
    """dict name -> (reference, error bound) in float64 of one sequence: q [n, hq, d], k, v [L, hk, d],
    seen [n] keys that each row sees."""
    n, hq, d = q.shape
    L, hk, _ = k.shape
    u = half_step(dtype)
    out = {}
    ke, ve = expand(k, hq), expand(v, hq)
    if L == 0:
        out["O"] = (np.zeros_like(q), np.zeros_like(q))
        out["lse"] = (np.full((n, hq), -np.inf), np.zeros((n, hq)))
        if dO is not None:
            out["dQ"] = (np.zeros_like(q), np.zeros_like(q))
            out["dK"] = out["dV"] = (np.zeros_like(k), np.zeros_like(k))
        return out
    mask = (np.arange(L)[None] < np.asarray(seen)[:, None])[:, None]  # [n, 1, L]
    S = np.einsum("nhd,lhd->nhl", q, ke) * scale
    mag = np.einsum("nhd,lhd->nhl", np.abs(q), np.abs(ke)) * abs(scale)
    e = np.where(mask, ES + 2.0 ** -23 * d * mag, 0.0).max(axis=2, keepdims=True)
    S = np.where(mask, S, -np.inf)
    m = S.max(axis=2, keepdims=True)
    ex = np.where(mask, np.exp(S - np.where(np.isfinite(m), m, 0.0)), 0.0)
    l = ex.sum(axis=2, keepdims=True)
    P = ex / np.where(l > 0, l, 1.0)
    with np.errstate(divide="ignore"):
        lse = np.where(l > 0, m + np.log(l), -np.inf)[..., 0]
    O = np.einsum("nhl,lhd->nhd", P, ve)
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    A = np.einsum("nhl,lhd->nhd", P, np.abs(ve))
    B = np.einsum("nhl,lhd->nhd", np.broadcast_to(mask, P.shape).astype(float), np.abs(ve))
    eO = 1.05 * ((u + 2 * e) * A + tiny * B)
    # a result below the 16-bit type's normal range rounds by half its smallest step
    least = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    out["O"] = (O, eO + u * np.abs(O) + least)
    out["lse"] = (lse, e[..., 0] + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0.0)))
    if dO is None:
        return out
    G = np.einsum("nhd,lhd->nhl", dO, ve)
    Gm = np.einsum("nhd,lhd->nhl", np.abs(dO), np.abs(ve))
    delta = (dO * O).sum(axis=2, keepdims=True)
    e_delta = (np.abs(dO) * (eO + u * np.abs(O) + least)).sum(axis=2, keepdims=True) \
        + 2.0 ** -23 * d * (np.abs(dO) * np.abs(O)).sum(axis=2, keepdims=True)
    dS = P * (G - delta) * scale
    e_dS = (np.abs(dS) * (u + 2 * e) + P * abs(scale) * (1 + 2 * e) * (e_delta + 2.0 ** -23 * d * Gm)) * 1.05 + tiny
    e_P = (P * (u + 2 * e)) * 1.05 + tiny

    def fold(x):  # [L, hq, d] -> [L, hk, d]
        return x.reshape(L, hk, hq // hk, d).sum(axis=2)

    dQ = np.einsum("nhl,lhd->nhd", dS, ke)
    out["dQ"] = (dQ, np.einsum("nhl,lhd->nhd", e_dS, np.abs(ke)) + u * np.abs(dQ) + least)
    dK = fold(np.einsum("nhl,nhd->lhd", dS, q))
    out["dK"] = (dK, fold(np.einsum("nhl,nhd->lhd", e_dS, np.abs(q))) + u * np.abs(dK) + least)
    dV = fold(np.einsum("nhl,nhd->lhd", P, dO))
    out["dV"] = (dV, fold(np.einsum("nhl,nhd->lhd", e_P, np.abs(dO))) + u * np.abs(dV) + least)
    return out


def check(name, got, ref, bound):
    got = got.detach().double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    fin = np.isfinite(ref)
    assert np.array_equal(got[~fin], ref[~fin]), "%s: infinities differ" % name
    assert np.isfinite(got[fin]).all(), "%s: not finite" % name
    over = np.abs(got[fin] - ref[fin]) - bound[fin]
    if over.size:
        assert over.max() <= 0, "%s: error %.3g over the bound %.3g" % (
            name, np.abs(got[fin] - ref[fin])[over.argmax()], bound[fin][over.argmax()])


def offsets(lens, device="cuda"):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=device)


def f64(t):
    return t.detach().double().cpu().numpy()
