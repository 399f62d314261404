"""The decoder layer's operators around the FP8 products, in FP64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The residual RMS norm with its FP8 output and gradient, the paged FP8 cache's
append and attention, and the few-token mixture-of-experts layer, each as the
plain loop over what it is defined on.
"""

import numpy as np

from . import e4m3, e5m2
from .gemm import bf16_rne
from .quant import BLOCK

_FORMATS = {"e4m3": (e4m3.E4M3_MAX, e4m3.encode_rne_sat, e4m3.decode),
            "e5m2": (e5m2.E5M2_MAX, e5m2.encode_rne_sat, e5m2.decode)}


# ------------------------------------------------------------------- norm
def rmsnorm(X, R, gain, eps, bf16):
    """(h, rstd, y) of X [M, K] and the residual R (or None); h is rounded to
    BF16 or FP32 when there is one."""
    h = np.asarray(X, dtype=np.float64)
    if R is not None:
        h = h + np.asarray(R, dtype=np.float64)
        h = bf16_rne(h) if bf16 else h.astype(np.float32).astype(np.float64)
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h, rstd, h * rstd[:, None] * np.asarray(gain, dtype=np.float64)


def rmsnorm_backward(dY, H, rstd, gain, dH=None):
    dY, H, gain = (np.asarray(a, dtype=np.float64) for a in (dY, H, gain))
    r = np.asarray(rstd, dtype=np.float64)[:, None]
    xhat = H * r
    dg = dY * gain
    dX = r * (dg - xhat * np.mean(dg * xhat, axis=1, keepdims=True))
    if dH is not None:
        dX = dX + np.asarray(dH, dtype=np.float64)
    return dX, np.sum(dY * xhat, axis=0)


# ------------------------------------------------------------------ cache
def pow2_scale(amax, limit):
    """Smallest power of two >= amax / limit (FP32 division), at least 2^-126."""
    q = float(np.float32(amax) / np.float32(limit))
    if q == 0.0 and amax == 0.0:
        return 0.0
    p = 2.0 ** -126
    while p < q:
        p *= 2.0
    return p


def kv_append(X, cache, scale, table, lens, cu, fmt="e4m3"):
    """New tokens X [T, heads, dim] into codes [blocks, heads, block, dim] and
    scales [blocks, heads], in place."""
    limit, encode, decode = _FORMATS[fmt]
    _, heads, block, _ = cache.shape
    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        start = int(lens[b]) - n
        for j in range(start // block, -(-int(lens[b]) // block)):
            r0, r1 = max(start - j * block, 0), min(int(lens[b]) - j * block, block)
            if r0 >= r1:
                continue
            blk = int(table[b, j])
            t = int(cu[b]) + j * block + r0 - start
            for h in range(heads):
                x = np.asarray(X[t:t + r1 - r0, h], dtype=np.float32)
                s = pow2_scale(np.max(np.abs(x)), limit)
                old = float(scale[blk, h])
                if r0 > 0:
                    s = max(s, old)
                    if s > old:
                        held = decode(cache[blk, h, :r0]) * (old / s)
                        cache[blk, h, :r0] = encode(held.astype(np.float32))
                if s > 0:
                    x = (x / np.float32(s)).astype(np.float32)
                cache[blk, h, r0:r1] = encode(x) if s > 0 else 0
                scale[blk, h] = s


def kv_attention(Q, kc, ks, vc, vs, table, lens, cu, scale, fmt="e4m3"):
    """(O, A) of Q [T, heads group, dim]: the outputs and the sums of
    p |v| that bound their rounding."""
    decode = _FORMATS[fmt][2]
    _, heads, block, dim = kc.shape
    group = Q.shape[1] // heads
    O = np.zeros(Q.shape)
    A = np.zeros(Q.shape)
    for b in range(len(lens)):
        L = int(lens[b])
        n = int(cu[b + 1] - cu[b])
        blocks = [int(x) for x in table[b, :-(-L // block)]]
        if not blocks:
            continue
        k = np.concatenate([decode(kc[x]) * ks[x].astype(np.float64)[:, None, None]
                            for x in blocks], axis=1)
        v = np.concatenate([decode(vc[x]) * vs[x].astype(np.float64)[:, None, None]
                            for x in blocks], axis=1)
        for i in range(n):
            sees = L - n + 1 + i
            if sees <= 0:
                continue
            t = int(cu[b]) + i
            for h in range(heads * group):
                x = scale * (k[h // group, :sees] @ Q[t, h].astype(np.float64))
                p = np.exp(x - np.max(x))
                p /= np.sum(p)
                O[t, h] = p @ v[h // group, :sees]
                A[t, h] = p @ np.abs(v[h // group, :sees])
    return O, A


def kv_attention_chunk(Q, kc, ks, vc, vs, table, lens, cu, scale, fmt="e4m3", causal=True):
    """kv_attention for many queries; causal=False: each sees the whole sequence.  NaN where no
    sequence has the row."""
    decode = _FORMATS[fmt][2]
    heads, block, dim = kc.shape[1:]
    group = Q.shape[1] // heads
    O, A = np.full(Q.shape, np.nan), np.full(Q.shape, np.nan)
    for b in range(len(lens)):
        L, t0, n = int(lens[b]), int(cu[b]), int(cu[b + 1] - cu[b])
        blocks = [int(x) for x in table[b, :-(-L // block)]]
        O[t0:t0 + n], A[t0:t0 + n] = 0.0, 0.0
        for h in range(heads):
            if not blocks:
                continue
            k, v = (np.concatenate([decode(c[x, h]) * np.float64(s[x, h]) for x in blocks])[:L]
                    for c, s in ((kc, ks), (vc, vs)))
            x = scale * np.einsum("ngd,ld->ngl", Q[t0:t0 + n, h * group:h * group + group].astype(np.float64), k)
            sees = L - n + 1 + np.arange(n) if causal else np.full(n, L)
            hidden = np.arange(L) >= sees[:, None, None]
            x = np.where(hidden, -np.inf, x)
            top = np.max(x, axis=2, keepdims=True)
            p = np.where(hidden, 0.0, np.exp(x - np.where(np.isneginf(top), 0, top)))
            p /= np.maximum(np.sum(p, axis=2, keepdims=True), 1e-300)
            O[t0:t0 + n, h * group:h * group + group] = np.einsum("ngl,ld->ngd", p, v)
            A[t0:t0 + n, h * group:h * group + group] = np.einsum("ngl,ld->ngd", p, np.abs(v))
    return O, A


# -------------------------------------------------------------------- MoE
def moe_route(logits, k, renormalise=True):
    logits = np.asarray(logits, dtype=np.float64)
    x = np.where(np.isnan(logits), -np.inf, logits)
    ids = np.argsort(-x, axis=1, kind="stable")[:, :k].astype(np.int32)
    top = np.take_along_axis(x, ids, 1)
    e = np.exp(top - top[:, :1])
    total = e.sum(1) if renormalise else np.exp(x - top[:, :1]).sum(1)
    return ids, e / total[:, None]


def _dequant(W, s):
    N, K = W.shape
    return e4m3.decode(W) * np.repeat(np.repeat(s.astype(np.float64), BLOCK, 0)[:N], BLOCK, 1)[:, :K]


def moe(A, sA, logits, W1, s1, W2, s2, k, renormalise=True):
    """(out, ids, weights); the hidden activations are quantised per 1x128
    block as FP32 values."""
    T, H = A.shape
    I = W2.shape[2]
    x = e4m3.decode(A) * np.repeat(sA.astype(np.float64), BLOCK, 1)[:, :H]
    ids, w = moe_route(logits, k, renormalise)
    out = np.zeros((T, H))
    for e in sorted(set(ids.ravel().tolist())):
        t, j = np.nonzero(ids == e)
        u = x[t] @ _dequant(W1[e], s1[e]).T
        gate, up = u[:, :I], u[:, I:]
        h = gate / (1.0 + np.exp(-gate)) * up
        for kb in range(-(-I // BLOCK)):
            blk = h[:, kb * BLOCK:(kb + 1) * BLOCK]
            s = np.max(np.abs(blk), axis=1, keepdims=True) / e4m3.E4M3_MAX
            q = e4m3.decode(e4m3.encode_rne_sat((blk / np.where(s > 0, s, 1)).astype(np.float32)))
            h[:, kb * BLOCK:(kb + 1) * BLOCK] = q * s
        np.add.at(out, t, w[t, j][:, None] * (h @ _dequant(W2[e], s2[e]).T))
    return out, ids, w


# --------------------------------------------------------- rotary positions
def rope(X, positions, freq, amplitude=1.0, interleaved=False, backward=False):
    """X [T, heads, dim] turned by positions [T] times freq [rot / 2]."""
    y = np.asarray(X, dtype=np.float64).copy()
    half = len(freq)
    t = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(freq, dtype=np.float64)
    c, s = amplitude * np.cos(t)[:, None], amplitude * np.sin(t)[:, None]
    if backward:
        s = -s
    i, j = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    a, b = y[..., i].copy(), y[..., j].copy()
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    return y


# ------------------------------------------------------- gated feed-forward
def gated(A, sA, W1, s1, a_fmt="e4m3"):
    """(h, u) of u = A W1^T [M, 2 I], h = silu(u[:, :I]) u[:, I:]."""
    x = _FORMATS[a_fmt][2](A) * np.repeat(sA.astype(np.float64), BLOCK, 1)[:, :A.shape[1]]
    u = x @ _dequant(W1, s1).T
    I = u.shape[1] // 2
    return u[:, :I] / (1.0 + np.exp(-u[:, :I])) * u[:, I:], u


def gated_backward(dY, sdY, W2T, s2T, GU, fmt="e5m2"):
    """(dgate, dup, dh) for dh = dY W2T^T and the gate and up values GU [M, 2 I]."""
    x = _FORMATS[fmt][2](dY) * np.repeat(sdY.astype(np.float64), BLOCK, 1)[:, :dY.shape[1]]
    dh = x @ _dequant(W2T, s2T).T
    I = dh.shape[1]
    g, u = GU[:, :I].astype(np.float64), GU[:, I:].astype(np.float64)
    s = 1.0 / (1.0 + np.exp(-g))
    return dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s, dh
