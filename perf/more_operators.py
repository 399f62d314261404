"""Measured cases of the operators that a decoder layer needs for prompts and for training.

  rope        rotary positions of queries and keys, forward and gradient
  chunk       attention of a chunk of new tokens (or of queries that see everything) over the paged FP8 cache
  gated       gate and up products in FP8, SwiGLU and the 1x128 quantiser in one pass (the producer of the down product)
  gated_grad  its gradient: the product with the down weight, SwiGLU's gradient and the quantiser

`run` computes them in elementary torch operations in 32 bits, or, where `own` is true, through the package.
"""
import math
import random

import torch

own = False

DEV = "cuda"
LIMIT = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
SCORES = 1 << 28  # scores that a plain attention holds at once


def listed():
    return [
        # one decode step of 64 sequences at far positions of long contexts: pure latency
        {"name": "rope_step", "op": "rope", "B": 64, "ctx": 131000, "new": 1, "hq": 64, "hk": 8, "dim": 128, "rot": 128,
         "layout": "half", "table": "ramp", "type": "bf16", "grad": False},
        # prompts of different lengths, queries and keys as parts of a fused projection's rows
        {"name": "rope_prompt", "op": "rope", "B": 5, "ctx": 700, "new": 4097, "hq": 64, "hk": 8, "dim": 128, "rot": 128,
         "layout": "half", "table": "linear", "type": "bf16", "grad": False},
        # a training micro-batch of 8192 tokens in packed documents, interleaved pairs in half of each head: the gradient
        {"name": "rope_grad", "op": "rope", "B": 7, "ctx": 0, "new": 2048, "hq": 32, "hk": 8, "dim": 128, "rot": 64,
         "layout": "interleaved", "table": "plain", "type": "bf16", "grad": True},
        # a chat's second message behind a short first one, one small head pair: the smallest call
        {"name": "chunk_short", "op": "chunk", "B": 1, "ctx": 37, "new": 17, "heads": 2, "group": 1, "dim": 64,
         "block": 16, "fmt": "e4m3", "causal": True},
        # a batch of ragged prompts with nothing before them, 64 query heads on 8 cached ones
        {"name": "chunk_prompts", "op": "chunk", "B": 9, "ctx": 0, "new": 4096, "heads": 8, "group": 8, "dim": 128,
         "block": 64, "fmt": "e4m3", "causal": True},
        # 512 more tokens of one long document
        {"name": "chunk_long", "op": "chunk", "B": 1, "ctx": 131077, "new": 512, "heads": 8, "group": 4, "dim": 128,
         "block": 64, "fmt": "e4m3", "causal": True},
        # a decoder's tokens on an encoder's states of another length, one head each
        {"name": "chunk_cross", "op": "chunk", "B": 8, "ctx": 1500, "new": 448, "heads": 16, "group": 1, "dim": 64,
         "block": 32, "fmt": "e5m2", "causal": False},
        # one decode token through a feed-forward block of the benchmark's sizes: the weights' bytes
        {"name": "gated_step", "op": "gated", "M": 1, "K": 7168, "I": 2048, "fmt": "e4m3", "save": False},
        # a few tokens, widths that are no multiples of the scale block
        {"name": "gated_odd", "op": "gated", "M": 77, "K": 1040, "I": 400, "fmt": "e4m3", "save": True},
        # a 4096-token prompt, the benchmark's prefill rows
        {"name": "gated_prompt", "op": "gated", "M": 4096, "K": 7168, "I": 2048, "fmt": "e4m3", "save": False},
        # a small model's micro-batch
        {"name": "gated_grad_small", "op": "gated_grad", "M": 130, "K": 400, "I": 272, "fmt": "e4m3", "save": True},
        # a training micro-batch of 8192 tokens, gradients in e5m2
        {"name": "gated_grad_train", "op": "gated_grad", "M": 8192, "K": 7168, "I": 2048, "fmt": "e5m2", "save": True},
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["rope", "rope", "chunk", "chunk", "chunk", "gated", "gated", "gated_grad"])
    if op == "rope":
        new = log(1, 4097)
        dim = rng.choice([64, 96, 128, 256])
        hk, group = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 4, 7, 8])
        kind = rng.choice(["bf16", "bf16", "f32"])
        most = 350000000 // ((group + 1) * hk * dim * (4 if kind == "bf16" else 8))  # tokens
        new = min(new, most)
        return {"op": op, "B": log(1, max(1, min(128, most // new))), "ctx": log(1, 131000), "new": new, "hq": hk * group,
                "hk": hk, "dim": dim, "rot": rng.choice([dim, dim, dim // 2 // 16 * 16]),
                "layout": rng.choice(["half", "interleaved"]), "table": rng.choice(["plain", "linear", "ramp"]),
                "type": kind, "grad": rng.random() < 0.4}
    if op == "chunk":
        new = log(1, 4097)
        heads, group = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 4, 5, 8])
        dim = rng.choice([64, 128])
        most = 1100000000000 // (4 * heads * group * dim)  # (query token, cached token) pairs
        ctx = log(1, min(131077, most // new - new))
        B = log(1, max(1, min(64, most // (new * (ctx + new)), 131072 // (ctx + new))))
        return {"op": op, "B": B, "ctx": ctx, "new": new, "heads": heads, "group": group, "dim": dim,
                "block": rng.choice([16, 32, 64, 128]), "fmt": rng.choice(["e4m3", "e4m3", "e5m2"]),
                "causal": rng.random() < 0.75}
    I = 16 * log(8, 256)
    K = 16 * log(16, 448)
    M = log(1, min(8192, max(64, 8192 * 2048 * 7168 // (I * K) // (2 if op == "gated" else 1))))
    return {"op": op, "M": M, "K": K, "I": I, "fmt": rng.choice(["e4m3", "e5m2"]), "save": rng.random() < 0.5}


# ---------------------------------------------------------------- sizes that follow from a case
def cached(case):
    """Tokens of each sequence in the cache before the call's own: ragged, the first one the longest."""
    r = random.Random(case["ctx"] * 1009 + case["B"])
    return [case["ctx"]] + [r.randint(case["ctx"] // 2, case["ctx"]) for _ in range(case["B"] - 1)]


def new_counts(case):
    r = random.Random(case["new"] * 31 + case["B"])
    return [case["new"]] + [r.randint(1, case["new"]) for _ in range(case["B"] - 1)]


def seen(case):
    """Tokens that each sequence's queries attend to (the last query's, where they are causal)."""
    return [a + n if case["causal"] else max(a, 1) for a, n in zip(cached(case), new_counts(case))]


def pairs(case):
    """Visible (query token, cached token) pairs."""
    total = 0
    for n, L in zip(new_counts(case), seen(case)):
        total += n * L - n * (n - 1) // 2 if case["causal"] else n * L
    return total


def ceil_div(a, b):
    return -(-a // b)


def offsets(counts):
    return [sum(counts[:i]) for i in range(len(counts) + 1)]


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- prepare
def frequencies(case):
    """Radians a position for each pair, and the amplitude: plain, all slowed down to reach four times the
    trained length, or only the slow ones (a ramp between the pairs that turn 32 times and once within it)."""
    half = case["rot"] // 2
    f = [10000.0 ** (-i / half) for i in range(half)]
    if case["table"] == "linear":
        return torch.tensor([x / 4 for x in f], device=DEV), 1.0
    if case["table"] == "ramp":
        keep = [min(1.0, max(0.0, math.log(max(8192 * x / (2 * math.pi), 1e-9)) / math.log(32))) for x in f]
        return torch.tensor([x * k + x / 16 * (1 - k) for x, k in zip(f, keep)], device=DEV), 0.1 * math.log(16) + 1
    return torch.tensor(f, device=DEV), 1.0


def prepare_rope(case, seed):
    g, t = gen(seed), TYPE[case["type"]]
    new = new_counts(case)
    T, hq, hk, D = sum(new), case["hq"], case["hk"], case["dim"]
    s = {}
    s["freq"], s["amplitude"] = frequencies(case)
    parts = [hq * D, hk * D, hk * D]
    fused = randn(g, T, sum(parts)).to(t)  # a fused projection's rows: queries, keys and values
    apart = [torch.empty((T, h, D), dtype=t, device=DEV) for h in (hq, hk)]
    view = [x.unflatten(1, (-1, D)) for x in fused.split(parts, 1)[:2]]
    if case["grad"]:  # gradients of the rotated ones, into the places of the projection's gradient
        apart = [randn(g, T, h, D).to(t) for h in (hq, hk)]
        s["q"], s["k"], s["qo"], s["ko"] = *apart, *view
        s["positions"] = i32([p for n in new for p in range(n)])
    else:
        s["q"], s["k"], s["qo"], s["ko"] = *view, *apart
        old = cached(case)
        s["lens"], s["cu"] = i32([a + n for a, n in zip(old, new)]), i32(offsets(new))
    return s


def paged(g, lens, heads, dim, block, fmt):
    """A cache that holds `lens` tokens of each sequence in blocks in no order, with stale numbers behind them."""
    per = [ceil_div(n, block) for n in lens]
    width, total = max(1, max(per)), max(1, sum(per)) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    used, starts = torch.tensor(per, device=DEV), torch.tensor(offsets(per)[:-1], device=DEV)
    col = torch.arange(width, device=DEV)
    at = (starts[:, None] + col).clamp(max=total - 1)
    s = {"table": torch.where(col < used[:, None], order[at], torch.zeros_like(order[at])), "lens": i32(lens)}
    for name in ("k", "v"):
        codes = torch.empty((total, heads, block, dim), dtype=torch.uint8, device=DEV)
        for b in range(0, total, 4096):
            part = codes[b:b + 4096]
            x = (LIMIT[fmt] / 5 * randn(g, *part.shape)).clamp(-LIMIT[fmt], LIMIT[fmt])
            part.copy_(x.to(F8[fmt]).view(torch.uint8))
        s[name + "c"] = codes
        e = torch.randint(-1, 2, (total, heads), generator=g, device=DEV) + round(math.log2(5 / LIMIT[fmt]))
        s[name + "s"] = torch.exp2(e.float())
    return s


def prepare_chunk(case, seed):
    g = gen(seed)
    new = new_counts(case)
    T, hq, D = sum(new), case["heads"] * case["group"], case["dim"]
    s = paged(g, seen(case), case["heads"], D, case["block"], case["fmt"])
    s["cu"] = i32(offsets(new))
    s["q"] = (2 * randn(g, T, hq, D)).to(torch.bfloat16)
    s["scale"] = 1 / math.sqrt(D)
    s["O"] = torch.empty_like(s["q"])
    return s


def quantised_weight(g, N, K):
    Nb, Kb = ceil_div(N, 128), ceil_div(K, 128)
    w = torch.zeros((Nb * 128, Kb * 128), device=DEV)
    w[:N, :K] = randn(g, N, K) / math.sqrt(K)
    t = w.view(Nb, 128, Kb, 128)
    scale = t.abs().amax((1, 3)) / 448
    codes = (t / scale[:, None, :, None]).to(F8["e4m3"]).view(torch.uint8).view(Nb * 128, Kb * 128)
    return codes[:N, :K].contiguous(), scale


def prepare_gated(case, seed):
    g = gen(seed)
    M, K, I = case["M"], case["K"], case["I"]
    s = {}
    x = randn(g, M, K) * (2 * randn(g, M, 1)).exp2()  # rows of different sizes
    grad = case["op"] == "gated_grad"
    s["A"], s["sA"] = quant_rows(x / 64 if grad else x, case["fmt"])
    s["A"] = s["A"].view(torch.uint8)
    s["W"], s["sW"] = quantised_weight(g, I if grad else 2 * I, K)
    Ip = 128 * ceil_div(I, 128)
    if grad:
        s["GU"] = (2 * randn(g, M, 2 * I)).to(torch.bfloat16)
        s["dGU"] = torch.empty((M, 2 * I), dtype=torch.bfloat16, device=DEV) if case["save"] else None
        s["Q"], s["sQ"] = torch.empty((M, 2 * Ip), dtype=torch.uint8, device=DEV), torch.empty((M, 2 * Ip // 128), device=DEV)
    else:
        s["GU"] = torch.empty((M, 2 * I), dtype=torch.bfloat16, device=DEV) if case["save"] else None
        s["Q"], s["sQ"] = torch.empty((M, I), dtype=torch.uint8, device=DEV), torch.empty((M, Ip // 128), device=DEV)
    return s


def prepare(case, seed):
    fn = {"rope": prepare_rope, "chunk": prepare_chunk, "gated": prepare_gated, "gated_grad": prepare_gated}[case["op"]]
    return {"case": case, **fn(case, seed)}


# ---------------------------------------------------------------- plain forms
def quant_rows(y, fmt):
    """1x128 quantisation of the last axis: codes of y's shape and a scale for each block (0 for a block of zeros)."""
    K = y.shape[-1]
    Kb = ceil_div(K, 128)
    t = torch.nn.functional.pad(y, (0, Kb * 128 - K)).unflatten(-1, (Kb, 128))
    s = t.abs().amax(-1) / LIMIT[fmt]
    q = torch.where(s[..., None] > 0, t / s[..., None], torch.zeros_like(t)).clamp(-LIMIT[fmt], LIMIT[fmt])
    return q.flatten(-2)[..., :K].contiguous().to(F8[fmt]), s


def dequant(codes, scale, fmt, rows_a_block):
    """The values of a matrix of codes, in 32 bits."""
    if rows_a_block > 1:
        scale = scale.repeat_interleave(rows_a_block, 0)[:codes.shape[0]]
    return codes.view(F8[fmt]).float() * scale.repeat_interleave(128, 1)[:, :codes.shape[1]]


def plain_rope(s):
    c = s["case"]
    if c["grad"]:
        pos = s["positions"].double()
    else:
        cu, lens = s["cu"].long(), s["lens"].long()
        t = torch.arange(s["q"].shape[0], device=DEV)
        seq = torch.searchsorted(cu, t, right=True) - 1
        pos = ((lens - (cu[1:] - cu[:-1]))[seq] + t - cu[seq]).double()
    angle = pos[:, None] * s["freq"].double()  # 32 bits would lose the angles of far positions
    cos, sin = (f(angle).float()[:, None, :] * s["amplitude"] for f in (torch.cos, torch.sin))
    if c["grad"]:
        sin = -sin
    half = c["rot"] // 2
    out = {}
    for name in ("q", "k"):
        x, y = s[name].float(), s[name + "o"]
        if c["layout"] == "half":
            a, b = x[..., :half], x[..., half:c["rot"]]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        else:
            a, b = x[..., :c["rot"]:2], x[..., 1:c["rot"]:2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        y.copy_(torch.cat((turned, x[..., c["rot"]:]), -1))
        out[name] = y
    return out


def plain_chunk(s):
    c = s["case"]
    Hk, G, D, block, fmt = c["heads"], c["group"], c["dim"], c["block"], c["fmt"]
    cu = offsets(new_counts(c))
    for b, L in enumerate(seen(c)):
        n = cu[b + 1] - cu[b]
        ids = s["table"][b, :ceil_div(L, block)].long()
        k, v = ((s[x + "c"][ids].view(F8[fmt]).float() * s[x + "s"][ids][..., None, None]).transpose(0, 1)
                .reshape(Hk, -1, D)[:, :L] for x in ("k", "v"))
        q = s["q"][cu[b]:cu[b + 1]].float().view(n, Hk, G, D).permute(1, 0, 2, 3)
        step = max(1, SCORES // (Hk * G * L))
        at = torch.arange(L, device=DEV)
        for i in range(0, n, step):
            m = min(step, n - i)
            x = torch.matmul(q[:, i:i + m].reshape(Hk, m * G, D), k.transpose(1, 2)) * s["scale"]
            if c["causal"]:
                limit = (L - n + 1 + i + torch.arange(m, device=DEV)).repeat_interleave(G)
                x = torch.where(at < limit[:, None], x, torch.full((), -math.inf, device=DEV))
            p = torch.exp(x - x.amax(-1, keepdim=True))
            o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
            s["O"][cu[b] + i:cu[b] + i + m] = o.view(Hk, m, G, D).transpose(0, 1).reshape(m, Hk * G, D)
    return s["O"]


def plain_gated(s):
    c = s["case"]
    I = c["I"]
    u = dequant(s["A"], s["sA"], c["fmt"], 1) @ dequant(s["W"], s["sW"], "e4m3", 128).t()
    gate, up = u[:, :I], u[:, I:]
    q, sq = quant_rows(gate / (1 + torch.exp(-gate)) * up, c["fmt"])
    out = {"q": q, "s": sq}
    if c["save"]:
        out["gu"] = u.to(torch.bfloat16)
    return out


def plain_gated_grad(s):
    c = s["case"]
    I = c["I"]
    dh = dequant(s["A"], s["sA"], c["fmt"], 1) @ dequant(s["W"], s["sW"], "e4m3", 128).t()
    gate, up = s["GU"][:, :I].float(), s["GU"][:, I:].float()
    sig = 1 / (1 + torch.exp(-gate))
    parts = [dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig]
    pad = 128 * ceil_div(I, 128) - I  # each half starts at a scale block of its own
    q, sq = quant_rows(torch.cat([torch.nn.functional.pad(x, (0, pad)) for x in parts], 1), c["fmt"])
    out = {"q": q, "s": sq}
    if c["save"]:
        out["dgu"] = torch.cat(parts, 1).to(torch.bfloat16)
    return out


# ---------------------------------------------------------------- the package's operators
def own_run(s):
    from fp8_fine_grained_e4m3_gb300 import binding as fp8
    c = s["case"]
    op = c["op"]
    if op == "rope":
        where = {"positions": s["positions"]} if c["grad"] else {"seq_lens": s["lens"], "cu": s["cu"]}
        q, k = fp8.fp8_rope(s["q"], s["k"], s["freq"], interleaved=c["layout"] == "interleaved",
                            amplitude=s["amplitude"], backward=c["grad"], Qo=s["qo"], Ko=s["ko"], **where)
        return {"q": q, "k": k}
    if op == "chunk":
        return fp8.fp8_kv_attention_chunk(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["lens"],
                                          cu_q=s["cu"], max_q=c["new"], scale=s["scale"], causal=c["causal"],
                                          fmt=c["fmt"], O=s["O"])
    if op == "gated":
        q, sq = fp8.fp8gemm_gated(s["A"], s["sA"], s["W"], s["sW"], a_fmt=c["fmt"], fmt=c["fmt"], GU=s["GU"],
                                  Q=s["Q"], sQ=s["sQ"])
        out = {"q": q.view(F8[c["fmt"]]), "s": sq}
        if c["save"]:
            out["gu"] = s["GU"]
        return out
    q, sq = fp8.fp8gemm_gated_backward(s["A"], s["sA"], s["W"], s["sW"], s["GU"], a_fmt=c["fmt"], fmt=c["fmt"],
                                       dGU=s["dGU"], Q=s["Q"], sQ=s["sQ"])
    out = {"q": q.view(F8[c["fmt"]]), "s": sq}
    if c["save"]:
        out["dgu"] = s["dGU"]
    return out


def run(state):
    if own:
        return own_run(state)
    return {"rope": plain_rope, "chunk": plain_chunk, "gated": plain_gated,
            "gated_grad": plain_gated_grad}[state["case"]["op"]](state)


# ---------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "rope":
        T, el = sum(new_counts(case)), 2 if case["type"] == "bf16" else 4
        n = T * (case["hq"] + case["hk"])
        return {"bytes": 2 * n * case["dim"] * el + 2 * case["rot"] + 4 * (T if case["grad"] else 2 * case["B"]),
                "flops": 3 * n * case["rot"]}
    if op == "chunk":
        T, hq, w = sum(new_counts(case)), case["heads"] * case["group"], case["heads"] * case["dim"]
        blocks = sum(ceil_div(L, case["block"]) for L in seen(case))
        return {"bytes": 2 * sum(seen(case)) * w + blocks * (4 + 8 * case["heads"]) + 4 * T * hq * case["dim"],
                "flops": 4 * pairs(case) * hq * case["dim"]}
    M, K, I = case["M"], case["K"], case["I"]
    Kb, Ib = ceil_div(K, 128), ceil_div(I, 128)
    if op == "gated":
        return {"bytes": M * (K + 4 * Kb) + 2 * I * K + M * (I + 4 * Ib) + (4 * M * I if case["save"] else 0),
                "flops": 4 * M * I * K}
    return {"bytes": M * (K + 4 * Kb) + I * K + 4 * M * I + 2 * M * (128 * Ib + 4 * Ib) + (4 * M * I if case["save"] else 0),
            "flops": 2 * M * I * K}


# ---------------------------------------------------------------- the definitions in 64 bits
def round8(x, fmt):
    """To the nearest value of the format, ties to even, saturating: by the spacing of the value's binade."""
    bits, emin = (3, -6) if fmt == "e4m3" else (2, -14)
    e = torch.frexp(x.abs())[1].clamp(min=emin + 1) - 1
    step = torch.ldexp(torch.ones_like(x), e - bits)
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


def values(codes, scale, fmt, rows):
    x = codes.view(F8[fmt]).double()
    for i in range(0, x.shape[0], rows):
        for j in range(scale.shape[1]):
            x[i:i + rows, 128 * j:128 * j + 128] *= (scale[i // rows, j] if rows > 1 else scale[i, j]).double()
    return x


def values_of_rows(codes, scale, fmt):
    x = codes.view(F8[fmt]).double()
    for j in range(scale.shape[1]):
        x[:, 128 * j:128 * j + 128] *= scale[:, j:j + 1].double()
    return x


def exact_rope(st):
    c = st["case"]
    if c["grad"]:
        pos = st["positions"].tolist()
    else:
        pos = [a + i for a, n in zip(cached(c), new_counts(c)) for i in range(n)]
    pos = torch.tensor(pos, dtype=torch.float64, device=DEV)
    turn = torch.polar(torch.full((), st["amplitude"], dtype=torch.float64, device=DEV).expand(len(pos), c["rot"] // 2),
                       torch.outer(pos, st["freq"].double()))[:, None]
    if c["grad"]:
        turn = turn.conj()
    out = {}
    for name in ("q", "k"):
        x = st[name].double()
        y = x.clone()
        first, second = ((slice(0, c["rot"] // 2), slice(c["rot"] // 2, c["rot"])) if c["layout"] == "half" else
                         (slice(0, c["rot"], 2), slice(1, c["rot"], 2)))
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
        y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
    return out


def exact_chunk(st):
    c = st["case"]
    Hk, G, D, block = c["heads"], c["group"], c["dim"], c["block"]
    new = new_counts(c)
    out = torch.zeros((sum(new), Hk * G, D), dtype=torch.float64, device=DEV)
    t = 0
    for b, (n, L) in enumerate(zip(new, seen(c))):
        blocks = st["table"][b, :ceil_div(L, block)].long()
        for h in range(Hk):
            k, v = ((st[x + "c"][blocks, h].view(F8[c["fmt"]]).double() * st[x + "s"][blocks, h].double()[:, None, None])
                    .reshape(-1, D)[:L] for x in ("k", "v"))
            step = max(1, (1 << 26) // (G * L))
            for i in range(0, n, step):
                m = min(step, n - i)
                q = st["q"][t + i:t + i + m, h * G:h * G + G].double()
                x = torch.einsum("mgd,nd->mgn", q, k) * st["scale"]
                if c["causal"]:
                    sees = L - n + i + torch.arange(m, device=DEV)  # the last token that a query sees
                    x.masked_fill_((torch.arange(L, device=DEV) > sees[:, None])[:, None], -math.inf)
                out[t + i:t + i + m, h * G:h * G + G] = torch.einsum("mgn,nd->mgd", torch.softmax(x, -1), v)
        t += n
    return out


def exact_gated(st):
    c = st["case"]
    I = c["I"]
    u = values_of_rows(st["A"], st["sA"], c["fmt"]) @ values(st["W"], st["sW"], "e4m3", 128).t()
    q, s = exact_rows8(torch.nn.functional.silu(u[:, :I]) * u[:, I:], c["fmt"])
    return {"q": q, "s": s, **({"gu": u} if c["save"] else {})}


def exact_gated_grad(st):
    c = st["case"]
    I = c["I"]
    dh = values_of_rows(st["A"], st["sA"], c["fmt"]) @ values(st["W"], st["sW"], "e4m3", 128).t()
    with torch.enable_grad():
        gu = st["GU"].double().requires_grad_()
        (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]).backward(dh)
    d = gu.grad
    (qg, sg), (qu, su) = exact_rows8(d[:, :I], c["fmt"]), exact_rows8(d[:, I:], c["fmt"])
    gap = torch.zeros((d.shape[0], 128 * ceil_div(I, 128) - I), dtype=torch.float64, device=DEV)
    return {"q": torch.cat((qg, gap, qu, gap), 1), "s": torch.cat((sg, su), 1), **({"dgu": d} if c["save"] else {})}


def exact(case, seed):
    if case["op"] == "chunk" and pairs(case) * case["heads"] * case["group"] * case["dim"] > 2e12:
        return None
    st = prepare(case, seed)
    return {"rope": exact_rope, "chunk": exact_chunk, "gated": exact_gated, "gated_grad": exact_gated_grad}[case["op"]](st)
