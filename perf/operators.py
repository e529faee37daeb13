"""The measured cases of the sequence-attention operators and their plain forms.

Five operators of the path that joins the interaction rows of an example (candidates, the
rows of H_w) to that user's behaviour sequence (the rows of H_s):

    xattn   cross attention of jagged query rows over jagged key / value rows (serving)
    train   the same with its gradients (one training step of the operator)
    write   quantising new behaviour tokens into a paged cache of 8-bit rows
    read    reading cached sequences back as 16-bit rows
    serve   attention of each sequence's newest tokens over its cached pages

Sequences lie one after another in [tokens, heads, d] tensors; `q_off` and `kv_off` hold
their B + 1 boundaries. Head h of the queries reads key head h // (hq // hkv).
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # the 2-layer workload's 64 interaction rows of 128 over behaviour sequences of up to 2048 events, some users with none
        {"name": "xattn_c2", "op": "xattn", "b": 128, "n_lo": 64, "n_hi": 64, "l_lo": 0, "l_hi": 2048, "hq": 4, "hkv": 2, "d": 128, "dtype": "bf16", "lens": 11},
        # the 8-layer workload's 512 rows of 160, one head, sequences of 1024 to 4096 events
        {"name": "xattn_c4", "op": "xattn", "b": 48, "n_lo": 512, "n_hi": 512, "l_lo": 1024, "l_hi": 4096, "hq": 1, "hkv": 1, "d": 160, "dtype": "bf16", "lens": 12},
        # one candidate each for three users with short histories: the latency of a call
        {"name": "xattn_one", "op": "xattn", "b": 3, "n_lo": 1, "n_hi": 1, "l_lo": 1, "l_hi": 250, "hq": 4, "hkv": 4, "d": 64, "dtype": "f16", "lens": 13},
        # a training step at the 2-layer shape with ragged candidates and shared key heads
        {"name": "train_c2", "op": "train", "b": 64, "n_lo": 32, "n_hi": 64, "l_lo": 1, "l_hi": 2048, "hq": 4, "hkv": 2, "d": 128, "dtype": "bf16", "lens": 14},
        # a training step at the 8-layer shape
        {"name": "train_c4", "op": "train", "b": 16, "n_lo": 512, "n_hi": 512, "l_lo": 512, "l_hi": 4096, "hq": 1, "hkv": 1, "d": 160, "dtype": "f16", "lens": 15},
        # a small odd training batch with users that have no history
        {"name": "train_odd", "op": "train", "b": 5, "n_lo": 1, "n_hi": 37, "l_lo": 0, "l_hi": 211, "hq": 6, "hkv": 3, "d": 32, "dtype": "bf16", "lens": 16},
        # whole histories of 16 users enter the cache at once
        {"name": "write_history", "op": "write", "b": 16, "n_lo": 1024, "n_hi": 4096, "l_lo": 0, "l_hi": 100, "hkv": 4, "d": 128, "dtype": "bf16", "page": 64, "lens": 17},
        # one new event for each of 24 users
        {"name": "write_step", "op": "write", "b": 24, "n_lo": 1, "n_hi": 1, "l_lo": 0, "l_hi": 700, "hkv": 2, "d": 160, "dtype": "f16", "page": 16, "lens": 18},
        # the cached histories of 16 users back as 16-bit rows
        {"name": "read_history", "op": "read", "b": 16, "l_lo": 1024, "l_hi": 4096, "hkv": 4, "d": 128, "dtype": "bf16", "page": 64, "bits": 8, "lens": 19},
        # three short histories out of a 16-bit cache
        {"name": "read_short", "op": "read", "b": 3, "l_lo": 0, "l_hi": 77, "hkv": 2, "d": 64, "dtype": "f16", "page": 16, "bits": 16, "lens": 20},
        # the newest event of 64 users over 8-bit caches of up to 15,000 events
        {"name": "serve_step", "op": "serve", "b": 64, "n_lo": 1, "n_hi": 1, "l_lo": 1, "l_hi": 15000, "hq": 8, "hkv": 2, "d": 128, "dtype": "bf16", "page": 64, "bits": 8, "causal": True, "lens": 21},
        # chunks of up to 512 new events over a 16-bit cache
        {"name": "serve_chunk", "op": "serve", "b": 8, "n_lo": 200, "n_hi": 512, "l_lo": 512, "l_hi": 4096, "hq": 8, "hkv": 2, "d": 128, "dtype": "bf16", "page": 32, "bits": 16, "causal": True, "lens": 22},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["xattn", "train", "write", "read", "serve"])
    case = {"op": op, "d": rng.choice([32, 64, 128, 160]), "dtype": rng.choice(["bf16", "f16"]), "lens": rng.randrange(1 << 30)}
    case["hkv"] = rng.choice([1, 2, 3, 4])
    if op in ("xattn", "train", "serve"):
        case["hq"] = case["hkv"] * rng.choice([1, 2, 4, 5])
    if op != "xattn" and op != "train":
        case["page"] = rng.choice([16, 32, 64, 128])
    if op in ("read", "serve"):
        case["bits"] = rng.choice([8, 16])
    if op in ("xattn", "train"):
        case["n_hi"] = _log(rng, 1, 512)
        case["n_lo"] = rng.choice([1, case["n_hi"], (case["n_hi"] + 1) // 2])
        case["l_hi"] = _log(rng, 1, 4096)
        case["l_lo"] = rng.choice([0, 1, (case["l_hi"] + 1) // 2])
        most = (100 << 20) if op == "xattn" else (33 << 20)
        room = most // (case["hq"] * case["n_hi"] * case["l_hi"])
    elif op == "write":
        case["n_hi"] = _log(rng, 1, 4096)
        case["n_lo"] = (case["n_hi"] + 2) // 3
        case["l_lo"], case["l_hi"] = 0, _log(rng, 1, 1000)
        room = (8 << 20) // (case["n_hi"] * case["hkv"] * max(1, case["d"] // 32))
    elif op == "read":
        case["l_hi"] = _log(rng, 1, 4096)
        case["l_lo"] = rng.choice([0, case["l_hi"] // 3])
        room = (8 << 20) // (case["l_hi"] * case["hkv"] * max(1, case["d"] // 32))
    else:
        case["n_hi"] = rng.choice([1, 1, _log(rng, 2, 512)])
        case["n_lo"] = (case["n_hi"] + 1) // 2
        case["l_hi"] = _log(rng, case["n_hi"], 15000 if case["n_hi"] < 32 else 4096)
        case["l_lo"] = max(1, case["l_hi"] // 8)
        case["causal"] = rng.choice([True, True, False])
        room = min((100 << 20) // (case["hq"] * case["n_hi"] * case["l_hi"]), (8 << 20) // (case["l_hi"] * case["hkv"] * max(1, case["d"] // 32)))
    case["b"] = _log(rng, 1, max(1, min(64, room)))
    return case


def _lens(case):
    """(new tokens or query rows, sequence lengths) of the case's sequences. A sequence of a cache holds its new tokens too."""
    rng = random.Random(case["lens"])
    n = [rng.randint(case.get("n_lo", 0), case.get("n_hi", 0)) for _ in range(case["b"])]
    kv = [rng.randint(case["l_lo"], case["l_hi"]) for _ in range(case["b"])]
    kv[0] = case["l_hi"]  # the longest is there
    if case["op"] == "write":
        kv = [a + b for a, b in zip(n, kv)]
    elif case["op"] == "serve":
        kv = [max(a, b) for a, b in zip(n, kv)]
    return n, kv


def _offsets(lens):
    at = [0]
    for x in lens:
        at.append(at[-1] + x)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, d, hkv = DTYPES[case["dtype"]], case["d"], case["hkv"]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dt)

    n, kv = _lens(case)
    state = {"case": case, "dt": dt, "max_q": max(n), "max_kv": max(kv), "total_kv": sum(kv)}
    if case["op"] in ("xattn", "train", "serve"):
        state["q"] = normal(sum(n), case["hq"], d)
        state["q_off"] = _offsets(n)
        state["out"] = torch.empty_like(state["q"])
    if case["op"] in ("xattn", "train"):
        state["k"] = normal(sum(kv), hkv, d)
        state["v"] = normal(sum(kv), hkv, d)
        state["kv_off"] = _offsets(kv)
        if case["op"] == "train":
            state["grad"] = normal(sum(n), case["hq"], d)
    else:
        page = case["page"]
        each = [-(-x // page) for x in kv]
        pages, wide = sum(each) + 5, max(1, max(each))
        state["lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        state["kv_off"] = _offsets(kv)
        ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.zeros(case["b"], wide, dtype=torch.int32, device="cuda")
        at = 0
        for i, e in enumerate(each):
            table[i, :e] = ids[at : at + e]
            at += e
        state["table"] = table
        # rows differ in size, as the rows of different events do
        rows = torch.exp(torch.randn(2, pages, hkv, page, 1, generator=gen, device="cuda"))
        filled = [torch.randn(pages, hkv, page, d, generator=gen, device="cuda") * rows[i] for i in range(2)]
        if case["op"] == "write":
            state["new_k"], state["new_v"] = normal(sum(n), hkv, d), normal(sum(n), hkv, d, scale=3.0)
            state["q_off"] = _offsets(n)
        if case.get("bits", 8) == 8:
            (state["ck"], state["ek"]), (state["cv"], state["ev"]) = (_quantised(x) for x in filled)
        else:
            state["ck"], state["cv"] = (x.to(dt) for x in filled)
    return state


def _quantised(x):
    """Rows of d values as e4m3 values of x / 2^e and the biased exponents e + 127: the least e with amax <= 448 * 2^e."""
    amax = x.float().abs().amax(-1)
    frac, power = torch.frexp(amax)  # amax = frac * 2^power, frac in [1/2, 1)
    e = power - 9 + (frac > E4M3_MAX / 512.0)
    e = torch.where(amax > 0, e, -127).clamp(-127, 127)
    y = (x.double() * _power(-e).unsqueeze(-1)).float()
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _power(e):
    """2^e in 64 bits, from the bits of its exponent."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _dequantised(values, exponents):
    return (values.double() * _power(exponents.int() - 127).unsqueeze(-1)).float()


# ------------------------------------------------------------------ the plain forms


def _rows(off, most):
    """[B, most] places of each sequence's rows, and which of them there are."""
    i = torch.arange(most, device=off.device)
    there = i < (off[1:] - off[:-1]).unsqueeze(1)
    return torch.where(there, off[:-1].unsqueeze(1) + i, 0).long(), there


def _pages(cache, table):
    """[B, tokens, hkv, d or nothing] of a cache in the order of each sequence."""
    x = cache[table.long()].transpose(2, 3)
    return x.reshape(x.shape[0], -1, *x.shape[3:])


def _by_head(x, heads):
    """[B, rows, hq, d] -> [B, heads, hq // heads * rows, d]"""
    b, n, h, d = x.shape
    return x.view(b, n, heads, h // heads, d).permute(0, 2, 3, 1, 4).reshape(b, heads, -1, d)


def _weights(q, k, mask, scale):
    s = (q @ k.transpose(-1, -2) * scale).masked_fill(~mask, float("-inf"))
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top > float("-inf"), top, 0.0))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, 1.0)


def _plain_attention(state, k, v, keys, causal):
    """q over padded k, v [B, L, hkv, d] float32 of which `keys` [B] are there; also what the gradients need."""
    case = state["case"]
    at, there = _rows(state["q_off"], state["max_q"])
    q = torch.where(there[..., None, None], state["q"][at].float(), 0.0)
    b, n, hq, d = q.shape
    hkv, length = case["hkv"], k.shape[1]
    qh, kh, vh = _by_head(q, hkv), _by_head(k, hkv), _by_head(v, hkv)
    col = torch.arange(length, device=q.device)
    seen = keys.view(b, 1, 1).expand(b, n, 1)
    if causal:
        new = there.sum(1).view(b, 1, 1)
        seen = torch.minimum(seen, keys.view(b, 1, 1) - new + 1 + torch.arange(n, device=q.device).view(1, n, 1))
    mask = (col < seen) & there.unsqueeze(-1)
    mask = mask.unsqueeze(1).expand(b, hq // hkv, n, length).reshape(b, 1, -1, length)
    p = _weights(qh, kh, mask, 1.0 / math.sqrt(d))
    return p @ vh, p, qh, kh, vh, at, there


def _back(x, hq, there):
    """[B, hkv, g * rows, d] -> the rows that there are, [tokens, hq, d]"""
    b, hkv, _, d = x.shape
    return x.view(b, hkv, hq // hkv, -1, d).permute(0, 3, 1, 2, 4).reshape(b, -1, hq, d)[there]


def _plain(state):
    case, dt = state["case"], state["dt"]
    op = case["op"]
    if op == "write":
        k8, ke = _quantised(state["new_k"])
        v8, ve = _quantised(state["new_v"])
        off, page = state["q_off"].long(), case["page"]
        token = torch.arange(k8.shape[0], device=k8.device)
        seq = torch.searchsorted(off[1:], token, right=True)
        pos = state["lens"].long()[seq] - off[seq + 1] + token
        where = (state["table"].long()[seq, pos // page], pos % page)
        for held, new in ((state["ck"], k8), (state["cv"], v8), (state["ek"], ke), (state["ev"], ve)):
            held.view(torch.uint8)[where[0], :, where[1]] = new.view(torch.uint8)
        return [state["ck"], state["ek"], state["cv"], state["ev"]]
    if op in ("read", "serve"):
        if case["bits"] == 8:
            k, v = _dequantised(state["ck"], state["ek"]), _dequantised(state["cv"], state["ev"])
        else:
            k, v = state["ck"].float(), state["cv"].float()
        k, v = _pages(k, state["table"]), _pages(v, state["table"])
        if op == "read":
            _, there = _rows(state["kv_off"], k.shape[1])
            return [k[there].to(dt), v[there].to(dt)]
        o, *_, there = _plain_attention(state, k, v, state["lens"], case["causal"])
        return _back(o, case["hq"], there).to(dt)
    at, there = _rows(state["kv_off"], max(1, state["max_kv"]))
    if state["total_kv"] == 0:
        k = torch.zeros(case["b"], 1, case["hkv"], case["d"], device="cuda")
        v = k
    else:
        k = torch.where(there[..., None, None], state["k"][at].float(), 0.0)
        v = torch.where(there[..., None, None], state["v"][at].float(), 0.0)
    o, p, qh, kh, vh, q_at, q_there = _plain_attention(state, k, v, there.sum(1), False)
    out = _back(o, case["hq"], q_there).to(dt)
    if op == "xattn":
        return out
    scale = 1.0 / math.sqrt(case["d"])
    g = _by_head(torch.where(q_there[..., None, None], state["grad"][q_at].float(), 0.0), case["hkv"])
    dv = p.transpose(-1, -2) @ g
    ds = p * (g @ vh.transpose(-1, -2) - (g * o).sum(-1, keepdim=True)) * scale
    dq = _back(ds @ kh, case["hq"], q_there)
    dk = (ds.transpose(-1, -2) @ qh).transpose(1, 2)[there]
    return [out, dq.to(dt), dk.to(dt), dv.transpose(1, 2)[there].to(dt)]


# ------------------------------------------------------------------ the framework's calls


def _own(state):
    import recsys_feature_interaction_b200 as wk

    case = state["case"]
    op = case["op"]
    if op in ("xattn", "train"):
        q, k, v, out = state["q"], state["k"], state["v"], state["out"]
        if "ws" not in state:  # a user's program keeps these from call to call
            need = wk.wk_xattn_workspace(q, k, case["b"], state["max_q"], state["max_kv"], backward=op == "train")
            state["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
            if op == "train":
                state["lse"] = torch.empty(q.shape[0], q.shape[1], device="cuda")
                state["grads"] = [torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)]
        wk.wk_xattn_forward(q, k, v, out, state["q_off"], state["kv_off"], state["max_q"], state["max_kv"], lse=state.get("lse"), workspace=state["ws"])
        if op == "xattn":
            return out
        wk.wk_xattn_backward(q, k, v, out, state["lse"], state["grad"], *state["grads"], state["q_off"], state["kv_off"], state["max_q"], state["max_kv"], workspace=state["ws"])
        return [out, *state["grads"]]
    cache = {"K": state["ck"], "V": state["cv"], "K_exp": state.get("ek"), "V_exp": state.get("ev")}
    if op == "write":
        wk.wk_cache_write(cache, state["new_k"], state["new_v"], state["q_off"], state["table"], state["lens"], state["max_q"])
        return [state["ck"], state["ek"], state["cv"], state["ev"]]
    if op == "read":
        if "rows" not in state:
            state["rows"] = [torch.empty(state["total_kv"], case["hkv"], case["d"], dtype=state["dt"], device="cuda") for _ in range(2)]
        wk.wk_cache_read(cache, state["table"], state["lens"], state["kv_off"], *state["rows"], state["max_kv"])
        return state["rows"]
    if "ws" not in state:
        state["ws"] = torch.empty(wk.wk_cache_attention_workspace(cache, state["q"], case["b"], state["max_q"], state["max_kv"]), dtype=torch.uint8, device="cuda")
    wk.wk_cache_attention(cache, state["q"], state["out"], state["q_off"], state["table"], state["lens"], state["max_q"], state["max_kv"], causal=case["causal"], workspace=state["ws"])
    return state["out"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without


def _pairs(case):
    """How many (query row, key) pairs of one head take part."""
    n, kv = _lens(case)
    if case.get("causal"):
        return sum(a * b - a * (a - 1) // 2 for a, b in zip(n, kv))
    return sum(a * b for a, b in zip(n, kv))


def work(case):
    n, kv = _lens(case)
    d, hkv, op = case["d"], case["hkv"], case["op"]
    small = 4 * (case["b"] + 1)
    if op == "write":
        return {"bytes": sum(n) * hkv * 2 * (2 * d + d + 1) + 3 * small, "flops": sum(n) * hkv * 2 * 2 * d}
    held = (d + 1) if case.get("bits", 16) == 8 else 2 * d
    if op == "read":
        return {"bytes": sum(kv) * hkv * 2 * (held + 2 * d) + 3 * small, "flops": sum(kv) * hkv * 2 * d}
    rows, pairs = sum(n) * case["hq"] * d * 2, _pairs(case) * case["hq"] * d * 2
    if op == "train":
        # q, k, v and the output's gradient in; the output and three gradients out; seven products need two, five of them the backward
        return {"bytes": 4 * rows + 4 * sum(kv) * hkv * d * 2 + 2 * small, "flops": 7 * pairs}
    return {"bytes": 2 * rows + 2 * sum(kv) * hkv * held + 3 * small, "flops": 2 * pairs}


# ------------------------------------------------------------------ the definition in 64 bits


def _exact_quantised(x):
    """One tensor of rows as (values of x / 2^e rounded to e4m3, e + 127), from the definition: e by search, rounding by the step at each size."""
    x = x.double()
    amax = x.abs().amax(-1)
    powers = torch.tensor([2.0**i for i in range(-127, 128)], dtype=torch.float64, device=x.device)
    e = torch.searchsorted(powers * E4M3_MAX, amax.contiguous()).clamp(max=254)  # the first power that holds amax
    y = x / powers[e].unsqueeze(-1)
    size = torch.searchsorted(powers, y.abs().clamp(min=2.0**-6), right=True) - 1  # the last power that y reaches
    step = powers[size - 3]
    return torch.round(y / step) * step, e.to(torch.uint8)  # torch.round takes ties to even


def exact(case, seed):
    state = prepare(case, seed)
    n, kv = _lens(case)
    d, hkv, op = case["d"], case["hkv"], case["op"]
    if op in ("write", "read", "serve"):
        page, table = case["page"], state["table"].tolist()
        if case.get("bits", 8) == 8:
            powers = torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64, device="cuda")
            ck = state["ck"].double() * powers[state["ek"].long()].unsqueeze(-1)
            cv = state["cv"].double() * powers[state["ev"].long()].unsqueeze(-1)
        else:
            ck, cv = state["ck"].double(), state["cv"].double()
    if op == "write":
        out = [state["ck"].double(), state["ek"].clone(), state["cv"].double(), state["ev"].clone()]
        new = [*_exact_quantised(state["new_k"]), *_exact_quantised(state["new_v"])]
        at = 0
        for b in range(case["b"]):
            where = torch.arange(kv[b] - n[b], kv[b], device="cuda")
            ids = torch.tensor(table[b], device="cuda")[where // page]
            for held, x in zip(out, new):
                held[ids, :, where % page] = x[at : at + n[b]]
            at += n[b]
        return out

    def cached(held, b):
        ids = torch.tensor(table[b][: -(-kv[b] // page)], dtype=torch.long, device="cuda")
        return held[ids].permute(0, 2, 1, 3).reshape(-1, hkv, d)[: kv[b]]

    if op == "read":
        return [torch.cat([cached(held, b) for b in range(case["b"])]) for held in (ck, cv)]
    group, outs, grads, q_at, kv_at = case["hq"] // hkv, [], [[], [], []], 0, 0
    for b in range(case["b"]):
        q = state["q"][q_at : q_at + n[b]].double()
        if op == "serve":
            k, v = cached(ck, b), cached(cv, b)
        else:
            k, v = (state[x][kv_at : kv_at + kv[b]].double() for x in ("k", "v"))
        if op == "train":
            q, k, v = (x.requires_grad_() for x in (q, k, v))
        if kv[b]:
            s = torch.einsum("nhd,lhd->hnl", q, k.repeat_interleave(group, 1)) / d**0.5
            if case.get("causal"):
                late = torch.arange(kv[b], device="cuda") > torch.arange(kv[b] - n[b], kv[b], device="cuda").unsqueeze(1)
                s = s.masked_fill(late, float("-inf"))
            o = torch.einsum("hnl,lhd->nhd", torch.softmax(s, -1), v.repeat_interleave(group, 1))
        else:
            o = q * 0.0
        if op == "train":
            o.backward(state["grad"][q_at : q_at + n[b]].double())
            for held, x in zip(grads, (q, k, v)):
                held.append(torch.zeros_like(x) if x.grad is None else x.grad)
        outs.append(o.detach())
        q_at, kv_at = q_at + n[b], kv_at + kv[b]
    if op == "train":
        return [torch.cat(outs), *(torch.cat(x) for x in grads)]
    return torch.cat(outs)
