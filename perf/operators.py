"""Measured cases of the operators that stand between the block-scaled FP8 products of a decoder layer.

  norm      residual addition, root-mean-square norm and 1x128 FP8 output in one pass (the producer of a GEMM's A)
  norm_grad its gradient: input, residual stream and gain
  append    new keys and values into a paged FP8 cache with one scale for each block of tokens and head
  attend    attention of the newest tokens over that cache
  moe       a whole mixture-of-experts layer for a few tokens: routing, gate/up product, SwiGLU, down product, sum

`run` computes them in elementary torch operations in 32 bits, or, where `own` is true, through the package.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
LIMIT = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode token of a 7168-wide model between two layers: pure latency
        {"name": "norm_step", "op": "norm", "M": 1, "K": 7168, "type": "bf16", "fmt": "e4m3", "residual": True},
        # a 4096-token prompt, the benchmark's prefill rows
        {"name": "norm_prompt", "op": "norm", "M": 4096, "K": 7168, "type": "bf16", "fmt": "e4m3", "residual": True},
        # a small FP32 head whose width is no multiple of the scale block
        {"name": "norm_grad_small", "op": "norm_grad", "M": 130, "K": 400, "type": "f32", "residual": False},
        # a training micro-batch of 8192 tokens
        {"name": "norm_grad_train", "op": "norm_grad", "M": 8192, "K": 4096, "type": "bf16", "residual": True},
        # one decode step of 64 sequences: a token each, at a different place of its block
        {"name": "append_step", "op": "append", "B": 64, "ctx": 1024, "new": 1, "heads": 8, "dim": 128, "block": 64,
         "fmt": "e4m3"},
        # prompts of different lengths entering the cache, some behind earlier chunks
        {"name": "append_prompt", "op": "append", "B": 5, "ctx": 700, "new": 4097, "heads": 8, "dim": 128, "block": 16,
         "fmt": "e4m3"},
        # a chat's first tokens, one small head pair: the smallest call
        {"name": "attend_short", "op": "attend", "B": 1, "ctx": 37, "q": 1, "heads": 2, "group": 1, "dim": 64,
         "block": 16, "fmt": "e4m3"},
        # a serving batch: 64 ragged sequences of up to 8192 tokens, 64 query heads on 8 cached ones
        {"name": "attend_batch", "op": "attend", "B": 64, "ctx": 8192, "q": 1, "heads": 8, "group": 8, "dim": 128,
         "block": 64, "fmt": "e4m3"},
        # one long document with four speculated tokens checked at once
        {"name": "attend_long", "op": "attend", "B": 1, "ctx": 131077, "q": 4, "heads": 8, "group": 4, "dim": 128,
         "block": 64, "fmt": "e4m3"},
        # a single user's token through 4 of 32 experts (the benchmark's expert sizes)
        {"name": "moe_one", "op": "moe", "T": 1, "H": 7168, "I": 2048, "E": 32, "k": 4},
        # a handful of tokens, small experts, widths that are no multiples of the scale block
        {"name": "moe_odd", "op": "moe", "T": 5, "H": 1040, "I": 400, "E": 9, "k": 2},
        # 64 sequences' tokens through all 32 experts
        {"name": "moe_batch", "op": "moe", "T": 64, "H": 7168, "I": 2048, "E": 32, "k": 4},
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["norm", "norm_grad", "append", "attend", "attend", "moe", "moe"])
    if op in ("norm", "norm_grad"):
        K = 16 * log(8, 1024)
        M = log(1, min(8192, 33554432 // K))
        c = {"op": op, "M": M, "K": K, "type": rng.choice(["bf16", "bf16", "f32"]), "residual": rng.random() < 0.7}
        if op == "norm":
            c["fmt"] = rng.choice(["e4m3", "e4m3", "e5m2"])
        return c
    if op == "append":
        new = log(1, 4097)
        return {"op": op, "B": log(1, max(1, min(128, 16384 // new))), "ctx": log(1, 2048), "new": new,
                "heads": rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 128]), "block": rng.choice([16, 32, 64, 128]),
                "fmt": rng.choice(["e4m3", "e4m3", "e5m2"])}
    if op == "attend":
        ctx = log(1, 131077)
        heads = rng.choice([1, 2, 4, 5, 8])
        return {"op": op, "B": log(1, max(1, min(128, 262144 // ctx))), "ctx": ctx, "q": log(1, 8), "heads": heads,
                "group": rng.choice([1, 2, 4, 5, 8]), "dim": rng.choice([64, 128]),
                "block": rng.choice([16, 32, 64, 128]), "fmt": rng.choice(["e4m3", "e4m3", "e5m2"])}
    E = log(4, 64)
    H, I = 16 * log(16, 448), 16 * log(8, 128)
    E = min(E, max(4, 32 * 7168 * 2048 // (H * I)))
    return {"op": "moe", "T": log(1, 64), "H": H, "I": I, "E": E, "k": rng.randint(1, min(8, E))}


# ---------------------------------------------------------------- sizes that follow from a case
def lengths(case):
    """Cached tokens of each sequence before the call's own tokens: ragged, the first one the longest."""
    r = random.Random(case["ctx"] * 1009 + case["B"])
    return [case["ctx"]] + [r.randint(0, case["ctx"]) for _ in range(case["B"] - 1)]


def new_counts(case):
    r = random.Random(case["new"] * 31 + case["B"])
    return [case["new"]] + [r.randint(1, case["new"]) for _ in range(case["B"] - 1)]


def ceil_div(a, b):
    return -(-a // b)


def pow2(e, dtype=torch.float32):
    """2^e of whole numbers e, exactly: by the exponent's bits."""
    if dtype == torch.float64:
        return ((e.long() + 1023) << 52).view(dtype)
    return ((e.int() + 127) << 23).view(dtype)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


# ---------------------------------------------------------------- prepare
def prepare_norm(case, seed):
    g, t = gen(seed), TYPE[case["type"]]
    M, K = case["M"], case["K"]
    s = {"x": randn(g, M, K).to(t), "gain": 1 + 0.1 * randn(g, K)}
    s["x"][:, torch.arange(0, K, 101, device=DEV)] *= 30  # the few wide channels of a residual stream
    s["r"] = (2 * randn(g, M, K)).to(t) if case["residual"] else None
    if case["op"] == "norm_grad":
        h = s["x"].float() + (s["r"].float() if case["residual"] else 0)
        s["h"] = h.to(t)
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
        s["dy"] = (0.01 * randn(g, M, K)).to(t)
        s["dh"] = (0.02 * randn(g, M, K)).to(t) if case["residual"] else None
        s["dx"] = torch.empty((M, K), dtype=t, device=DEV)
        s["dgain"] = torch.empty(K, device=DEV)
        return s
    Kb = ceil_div(K, 128)
    s["Q"] = torch.empty((M, K), dtype=torch.uint8, device=DEV)
    s["sQ"] = torch.empty((M, Kb), device=DEV)
    s["H"] = torch.empty((M, K), dtype=t, device=DEV) if case["residual"] else None
    s["rstd"] = torch.empty(M, device=DEV)
    return s


def paged(g, lens, heads, dim, block, fmt):
    """A cache that holds `lens` tokens of each sequence in blocks in no order, with stale numbers behind them."""
    per = [ceil_div(n, block) for n in lens]
    width, total = max(1, max(per)), max(1, sum(per)) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    used, starts = torch.tensor(per, device=DEV), torch.tensor([sum(per[:i]) for i in range(len(per))], device=DEV)
    col = torch.arange(width, device=DEV)
    at = (starts[:, None] + col).clamp(max=total - 1)
    table = torch.where(col < used[:, None], order[at], torch.zeros_like(order[at]))
    s = {"table": table.contiguous(), "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    for name in ("k", "v"):
        codes = torch.empty((total, heads, block, dim), dtype=torch.uint8, device=DEV)
        for b in range(0, total, 4096):
            part = codes[b:b + 4096]
            x = (LIMIT[fmt] / 5 * randn(g, *part.shape)).clamp(-LIMIT[fmt], LIMIT[fmt])
            part.copy_(x.to(F8[fmt]).view(torch.uint8))
        s[name + "c"] = codes
        e = torch.randint(-1, 2, (total, heads), generator=g, device=DEV) + round(math.log2(5 / LIMIT[fmt]))
        s[name + "s"] = pow2(e)
    return s


def prepare_append(case, seed):
    g = gen(seed)
    old, new = lengths(case), new_counts(case)
    s = paged(g, [a + b for a, b in zip(old, new)], case["heads"], case["dim"], case["block"], case["fmt"])
    T, w = sum(new), case["heads"] * case["dim"]
    qkv = randn(g, T, 3 * w).to(torch.bfloat16)  # a fused projection's output; keys and values are parts of its rows
    s["k"], s["v"] = (qkv[:, i * w:(i + 1) * w].unflatten(1, (case["heads"], case["dim"])) for i in (1, 2))
    s["cu"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=DEV)
    return s


def prepare_attend(case, seed):
    g = gen(seed)
    lens = [n + case["q"] for n in lengths(case)]
    s = paged(g, lens, case["heads"], case["dim"], case["block"], case["fmt"])
    hq = case["heads"] * case["group"]
    s["q"] = (2 * randn(g, case["B"] * case["q"], hq, case["dim"])).to(torch.bfloat16)
    s["scale"] = 1 / math.sqrt(case["dim"])
    s["O"] = torch.empty_like(s["q"])
    return s


def quantised_weights(g, E, N, K):
    Nb, Kb = ceil_div(N, 128), ceil_div(K, 128)
    codes = torch.empty((E, N, K), dtype=torch.uint8, device=DEV)
    scale = torch.empty((E, Nb, Kb), device=DEV)
    for e in range(E):
        w = torch.zeros((Nb * 128, Kb * 128), device=DEV)
        w[:N, :K] = 0.02 * randn(g, N, K)
        t = w.view(Nb, 128, Kb, 128)
        scale[e] = t.abs().amax((1, 3)) / 448
        codes[e] = (t / scale[e][:, None, :, None]).to(F8["e4m3"]).view(torch.uint8).view(Nb * 128, Kb * 128)[:N, :K]
    return codes, scale


def prepare_moe(case, seed):
    g = gen(seed)
    T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
    s = {"logits": 2 * randn(g, T, E)}
    s["A"], s["sA"] = quant_rows(randn(g, T, H), "e4m3")
    s["A"] = s["A"].view(torch.uint8)
    s["W1"], s["s1"] = quantised_weights(g, E, 2 * I, H)
    s["W2"], s["s2"] = quantised_weights(g, E, H, I)
    s["D"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    s["ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
    s["w"] = torch.empty((T, k), device=DEV)
    return s


def prepare(case, seed):
    fn = {"norm": prepare_norm, "norm_grad": prepare_norm, "append": prepare_append, "attend": prepare_attend,
          "moe": prepare_moe}[case["op"]]
    return {"case": case, **fn(case, seed)}


# ---------------------------------------------------------------- plain forms
def to8(x, fmt):
    return x.clamp(-LIMIT[fmt], LIMIT[fmt]).to(F8[fmt])


def quant_rows(y, fmt):
    """1x128 quantisation of the last axis: codes of y's shape and a scale for each block (0 for a block of zeros)."""
    K = y.shape[-1]
    Kb = ceil_div(K, 128)
    t = torch.nn.functional.pad(y, (0, Kb * 128 - K)).unflatten(-1, (Kb, 128))
    s = t.abs().amax(-1) / LIMIT[fmt]
    q = torch.where(s[..., None] > 0, t / s[..., None], torch.zeros_like(t))
    return to8(q.flatten(-2)[..., :K].contiguous(), fmt), s


def spread(s, rows, cols, br):
    """A scale for each element from one for each br x 128 block."""
    if br > 1:
        s = s.repeat_interleave(br, -2)[..., :rows, :]
    return s.repeat_interleave(128, -1)[..., :cols]


def plain_norm(s):
    c = s["case"]
    h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["x"].dtype)
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(1) + EPS)
    q, sq = quant_rows(hf * rstd[:, None] * s["gain"], c["fmt"])
    return {"q": q, "s": sq, "h": h, "rstd": rstd}


def plain_norm_grad(s):
    dy, xhat = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
    dg = dy * s["gain"]
    dx = (dg - xhat * (dg * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["h"].dtype), "dgain": (dy * xhat).sum(0)}


def pow2_scale(amax, fmt):
    """The smallest power of two that is at least amax / limit (2^-126 at least; 0 for 0)."""
    m, e = torch.frexp(amax / LIMIT[fmt])
    e = torch.where(m == 0.5, e - 1, e).clamp(min=-126)
    return torch.where(amax > 0, pow2(e), torch.zeros_like(amax))


def plain_append(s):
    block, table = s["case"]["block"], s["table"].long()
    cu, lens = s["cu"].long(), s["lens"].long()
    t = torch.arange(s["k"].shape[0], device=DEV)
    seq = torch.searchsorted(cu, t, right=True) - 1
    pos = (lens - (cu[1:] - cu[:-1]))[seq] + t - cu[seq]
    blk, off = table[seq, pos // block], pos % block
    out = {}
    for name in ("k", "v"):
        out[name], out[name + "_scale"] = plain_append_one(s[name].float(), s[name + "c"], s[name + "s"],
                                                           s["case"]["fmt"], blk, off)
    return out


def plain_append_one(x, cache, scale, fmt, blk, off):
    total, heads, block, _ = cache.shape
    amax = torch.zeros((total, heads), device=DEV).index_reduce_(0, blk, x.abs().amax(-1), "amax")
    held = torch.full((total,), block, device=DEV).index_reduce_(0, blk, off, "amin")  # rows that stay in each block
    need = pow2_scale(amax, fmt)  # 0 for a block that gets no token
    s_new = torch.where((held == 0)[:, None], need, torch.maximum(scale, need))
    ratio = torch.where(s_new > 0, scale / s_new, torch.ones_like(scale))[:, :, None, None]
    stays = (torch.arange(block, device=DEV) < held[:, None])[:, None, :, None]
    cache.copy_(torch.where(stays, to8(cache.view(F8[fmt]).float() * ratio, fmt).view(torch.uint8), cache))
    scale.copy_(s_new)
    st = s_new[blk][:, :, None]
    cache[blk, :, off] = to8(torch.where(st > 0, x / st, torch.zeros_like(x)), fmt).view(torch.uint8)
    return cache.view(F8[fmt]), scale


def plain_attend(s):
    c = s["case"]
    B, L, Hk, G, D = c["B"], c["q"], c["heads"], c["group"], c["dim"]
    t, fmt = s["table"].long(), c["fmt"]
    N = t.shape[1] * c["block"]
    k = (s["kc"][t].view(F8[fmt]).float() * s["ks"][t][..., None, None]).transpose(1, 2).reshape(B, Hk, N, D)
    v = (s["vc"][t].view(F8[fmt]).float() * s["vs"][t][..., None, None]).transpose(1, 2).reshape(B, Hk, N, D)
    lens = s["lens"].long()
    at = torch.arange(N, device=DEV)
    v = torch.where((at < lens[:, None])[:, None, :, None], v, torch.zeros_like(v))
    q = s["q"].float().view(B, L, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, L * G, D)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    limit = (lens[:, None] - L + 1 + torch.arange(L, device=DEV)).repeat_interleave(G, 1)  # tokens a row sees
    seen = at < limit[:, None, :, None]
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(z > 0, z, torch.ones_like(z))
    return o.view(B, Hk, L, G, D).permute(0, 2, 1, 3, 4).reshape(B * L, Hk * G, D).to(torch.bfloat16)


def plain_moe(s):
    T, H, I, E, k = (s["case"][n] for n in ("T", "H", "I", "E", "k"))
    ids = torch.sort(s["logits"], dim=1, descending=True, stable=True).indices[:, :k]
    top = torch.gather(s["logits"], 1, ids)
    w = torch.exp(top - top[:, :1])
    w = w / w.sum(1, keepdim=True)
    x = s["A"].view(F8["e4m3"]).float() * spread(s["sA"], T, H, 1)
    few = T * k <= E  # the chosen experts alone, a copy for each choice; otherwise every expert with every token
    if few:
        pick = ids.flatten()
        rows = x.repeat_interleave(k, 0)[:, None, :]
    else:
        pick = torch.arange(E, device=DEV)
        rows = x.expand(E, T, H)
    w1 = s["W1"][pick].view(F8["e4m3"]).float() * spread(s["s1"][pick], 2 * I, H, 128)
    gu = torch.bmm(rows, w1.transpose(1, 2))
    gate, up = gu[..., :I], gu[..., I:]
    h8, hs = quant_rows(gate / (1 + torch.exp(-gate)) * up, "e4m3")
    h = h8.float() * spread(hs, 0, I, 1)
    w2 = s["W2"][pick].view(F8["e4m3"]).float() * spread(s["s2"][pick], H, I, 128)
    y = torch.bmm(h, w2.transpose(1, 2))
    if few:
        out = (y.view(T, k, H) * w[:, :, None]).sum(1)
    else:
        coef = torch.zeros((T, E), device=DEV).scatter_(1, ids, w)
        out = (y * coef.t()[:, :, None]).sum(0)
    return {"out": out.to(torch.bfloat16), "ids": ids.to(torch.int32), "w": w}


# ---------------------------------------------------------------- the package's operators
def own_run(s):
    from fp8_fine_grained_e4m3_gb300 import binding as fp8
    c = s["case"]
    op = c["op"]
    if op == "norm":
        q, sq, h, rstd = fp8.fp8_rmsnorm_quant(s["x"], s["gain"], EPS, residual=s["r"], fmt=c["fmt"], H=s["H"],
                                               Q=s["Q"], sQ=s["sQ"], rstd=s["rstd"])
        return {"q": q.view(F8[c["fmt"]]), "s": sq, "h": h, "rstd": rstd}
    if op == "norm_grad":
        dx, dgain = fp8.fp8_rmsnorm_backward(s["dy"], s["h"], s["rstd"], s["gain"], dH=s["dh"], dX=s["dx"],
                                             dgain=s["dgain"])
        return {"dx": dx, "dgain": dgain}
    if op == "append":
        fp8.fp8_kv_append(s["k"], s["v"], s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["lens"], cu_new=s["cu"],
                          max_new=c["new"], fmt=c["fmt"])
        return {"k": s["kc"].view(F8[c["fmt"]]), "k_scale": s["ks"], "v": s["vc"].view(F8[c["fmt"]]), "v_scale": s["vs"]}
    if op == "attend":
        return fp8.fp8_kv_attention(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["lens"],
                                    scale=s["scale"], fmt=c["fmt"], O=s["O"])
    out, ids, w = fp8.fp8_moe_few(s["A"], s["sA"], s["logits"], s["W1"], s["s1"], s["W2"], s["s2"], c["k"], D=s["D"],
                                  ids=s["ids"], weights=s["w"])
    return {"out": out, "ids": ids, "w": w}


def run(state):
    if own:
        return own_run(state)
    return {"norm": plain_norm, "norm_grad": plain_norm_grad, "append": plain_append, "attend": plain_attend,
            "moe": plain_moe}[state["case"]["op"]](state)


# ---------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        M, K, b = case["M"], case["K"], 2 if case["type"] == "bf16" else 4
        if op == "norm":  # x, r in; h, codes, scales, rstd out
            per = b * (3 if case["residual"] else 1) + 1
            return {"bytes": M * K * per + M * 4 * (ceil_div(K, 128) + 1) + 4 * K, "flops": 6 * M * K}
        per = b * (4 if case["residual"] else 3)  # dy, h (and dh) in; dx out
        return {"bytes": M * K * per + 4 * M + 8 * K, "flops": 10 * M * K}
    if op == "append":  # keys and values in, codes out; a scale read and written for each touched block and head
        new, old = new_counts(case), lengths(case)
        T, w = sum(new), case["heads"] * case["dim"]
        touched = sum((a + n - 1) // case["block"] - a // case["block"] + 1 for a, n in zip(old, new))
        return {"bytes": 2 * T * w * 3 + 2 * touched * case["heads"] * 8 + 8 * touched, "flops": 2 * T * w * 3}
    if op == "attend":
        toks = sum(n + case["q"] for n in lengths(case))
        hq, w = case["heads"] * case["group"], case["heads"] * case["dim"]
        blocks = sum(ceil_div(n + case["q"], case["block"]) for n in lengths(case))
        return {"bytes": 2 * toks * w + blocks * (4 + 8 * case["heads"]) + 4 * case["B"] * case["q"] * hq * case["dim"],
                "flops": 4 * toks * case["q"] * hq * case["dim"]}
    T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
    active = E * (1 - (1 - k / E) ** T)  # distinct experts that T tokens are expected to choose
    return {"bytes": active * 3 * H * I * (1 + 4 / 16384) + T * H * 3 + T * E * 4 + T * k * 8,
            "flops": 6 * T * k * H * I}


# ---------------------------------------------------------------- the definitions in 64 bits
def round8(x, fmt):
    """To the nearest value of the format, ties to even, saturating: by the spacing of the value's binade."""
    bits, emin = (3, -6) if fmt == "e4m3" else (2, -14)
    e = torch.frexp(x.abs())[1].clamp(min=emin + 1) - 1
    step = pow2(e - bits, torch.float64)
    return (torch.round(x / step) * step).clamp(-LIMIT[fmt], LIMIT[fmt])


def exact_rows8(y, fmt):
    """Values and scales of the 1x128 blocks of a matrix's rows."""
    q = torch.zeros_like(y)
    s = torch.zeros((y.shape[0], ceil_div(y.shape[1], 128)), dtype=torch.float64, device=DEV)
    for kb in range(s.shape[1]):
        part = y[:, 128 * kb:128 * kb + 128]
        s[:, kb] = part.abs().max(1).values / LIMIT[fmt]
        q[:, 128 * kb:128 * kb + 128] = round8(part / torch.where(s[:, kb] > 0, s[:, kb], 1.0)[:, None], fmt)
    return q, s


def exact_norm(st):
    c = st["case"]
    h = st["x"] if st["r"] is None else (st["x"].double() + st["r"].double()).to(st["x"].dtype)
    h64 = h.double()
    rstd = 1 / torch.sqrt((h64 * h64).sum(1) / c["K"] + EPS)
    q, s = exact_rows8(h64 * rstd[:, None] * st["gain"].double(), c["fmt"])
    return {"q": q, "s": s, "h": h64, "rstd": rstd}


def exact_norm_grad(st):
    K = st["case"]["K"]
    dy, h, g, r = st["dy"].double(), st["h"].double(), st["gain"].double(), st["rstd"].double()[:, None]
    inner = (dy * g * h).sum(1, keepdim=True)
    dx = r * dy * g - r ** 3 / K * inner * h
    if st["dh"] is not None:
        dx = dx + st["dh"].double()
    return {"dx": dx, "dgain": (dy * h * r).sum(0)}


def exact_append(st):
    c, fmt, block = st["case"], st["case"]["fmt"], st["case"]["block"]
    out = {}
    new, old = new_counts(c), lengths(c)
    for name in ("k", "v"):
        val = st[name + "c"].view(F8[fmt]).double()
        scale = st[name + "s"].double().clone()
        x = st[name].double()
        table = st["table"].tolist()
        t0 = 0
        for b, n in enumerate(new):
            pos = old[b]
            while pos < old[b] + n:
                i, off = divmod(pos, block)
                m = min(block - off, old[b] + n - pos)
                rows = x[t0:t0 + m].transpose(0, 1)  # [heads, m, dim]
                amax = rows.abs().amax((1, 2)) / LIMIT[fmt]
                low = pow2((torch.frexp(amax)[1] - 1).clamp(min=-126), torch.float64)
                need = torch.where(amax > 0, torch.where(amax > low, 2 * low, low), 0.0)
                blk = table[b][i]
                s = need if off == 0 else torch.maximum(need, scale[blk])
                div = torch.where(s > 0, s, 1.0)[:, None, None]
                if off:
                    val[blk, :, :off] = round8(val[blk, :, :off] * scale[blk][:, None, None] / div, fmt)
                val[blk, :, off:off + m] = round8(rows / div, fmt)
                scale[blk] = s
                pos, t0 = pos + m, t0 + m
        out[name], out[name + "_scale"] = val, scale
    return out


def exact_attend(st):
    c = st["case"]
    L, Hk, G, D, block = c["q"], c["heads"], c["group"], c["dim"], c["block"]
    out = torch.zeros((c["B"] * L, Hk * G, D), dtype=torch.float64, device=DEV)
    for b, n in enumerate(st["lens"].tolist()):
        blocks = st["table"][b, :ceil_div(n, block)].long()
        k, v = (st[x + "c"][blocks].view(F8[c["fmt"]]).double() * st[x + "s"][blocks].double()[..., None, None]
                for x in ("k", "v"))
        k, v = (y.permute(1, 0, 2, 3).reshape(Hk, -1, D)[:, :n] for y in (k, v))
        for i in range(L):
            sees = n - L + 1 + i
            if sees <= 0:
                continue
            q = st["q"][b * L + i].double().view(Hk, G, D)
            p = torch.softmax(torch.einsum("hgd,hnd->hgn", q, k[:, :sees]) * st["scale"], -1)
            out[b * L + i] = torch.einsum("hgn,hnd->hgd", p, v[:, :sees]).reshape(Hk * G, D)
    return out


def exact_moe(st):
    T, H, I, E, k = (st["case"][n] for n in ("T", "H", "I", "E", "k"))

    def weights(codes, scale):
        w = codes.view(F8["e4m3"]).double()
        for i in range(scale.shape[0]):
            w[128 * i:128 * i + 128] *= scale[i].double().repeat_interleave(128)[:w.shape[1]]
        return w

    x = st["A"].view(F8["e4m3"]).double()
    x = x * st["sA"].double().repeat_interleave(128, 1)[:, :H]
    ids = torch.zeros((T, k), dtype=torch.int32, device=DEV)
    w = torch.zeros((T, k), dtype=torch.float64, device=DEV)
    for t, row in enumerate(st["logits"].double().tolist()):
        best = sorted(range(E), key=lambda e: (-row[e], e))[:k]
        z = [math.exp(row[e] - row[best[0]]) for e in best]
        ids[t] = torch.tensor(best, dtype=torch.int32)
        w[t] = torch.tensor(z, dtype=torch.float64) / sum(z)
    out = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    for e in sorted(set(ids.flatten().tolist())):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gu = x[t] @ weights(st["W1"][e], st["s1"][e]).t()
        q, s = exact_rows8(torch.nn.functional.silu(gu[:, :I]) * gu[:, I:], "e4m3")
        h = q * s.repeat_interleave(128, 1)[:, :I]
        out.index_add_(0, t, w[t, j][:, None] * (h @ weights(st["W2"][e], st["s2"][e]).t()))
    return {"out": out, "ids": ids, "w": w}


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": exact_norm, "norm_grad": exact_norm_grad, "append": exact_append, "attend": exact_attend,
            "moe": exact_moe}[case["op"]](st)
