"""The oracle's rotary positions, chunk attention and gated block against other ways to the same numbers.  CPU only."""

import math

import numpy as np
import pytest

from oracle import layer
from oracle import quant as oq


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_complex_product(interleaved):
    g = np.random.default_rng(0)
    x, pos, f = g.standard_normal((5, 2, 12)), np.array([0, 1, 7, 1000, -3]), np.array([1.0, 0.3, 0.01])
    y = layer.rope(x, pos, f, 1.5, interleaved)
    i, j = (slice(0, 6, 2), slice(1, 6, 2)) if interleaved else (slice(0, 3), slice(3, 6))
    z = (x[..., i] + 1j * x[..., j]) * (1.5 * np.exp(1j * pos[:, None] * f))[:, None]
    assert np.allclose(y[..., i], z.real) and np.allclose(y[..., j], z.imag)
    assert np.array_equal(y[..., 6:], x[..., 6:]) and np.allclose(y[0, :, :6], 1.5 * x[0, :, :6])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient_is_the_adjoint(interleaved):
    g = np.random.default_rng(1)
    x, w = g.standard_normal((2, 6, 3, 16))
    args = (g.integers(0, 9999, 6), [1.0, 0.5, 0.1, 0.01], 1.2, interleaved)
    assert math.isclose(np.sum(w * layer.rope(x, *args)), np.sum(layer.rope(w, *args, backward=True) * x), rel_tol=1e-12)


@pytest.mark.parametrize("causal", [True, False])
def test_chunk_attention_token_by_token(causal):
    g = np.random.default_rng(2)
    heads, group, dim, block, lens, counts = 2, 2, 8, 4, [9, 3, 5], [4, 5, 2]
    kc, vc = (layer.e4m3.encode_rne_sat(g.standard_normal((6, heads, block, dim)).astype(np.float32)) for _ in range(2))
    ks, vs = (2.0 ** g.integers(-2, 3, (6, heads)).astype(np.float32) for _ in range(2))
    table = np.array([[0, 1, 2], [3, 0, 0], [4, 5, 0]])
    cu = np.concatenate([[0], np.cumsum(counts)])
    Q = g.standard_normal((sum(counts), heads * group, dim))
    O, A = layer.kv_attention_chunk(Q, kc, ks, vc, vs, table, lens, cu, 0.4, causal=causal)
    if causal:
        ref, size = layer.kv_attention(Q, kc, ks, vc, vs, table, lens, cu, 0.4)
    else:  # each query by itself, as the only new token
        ref, size = np.zeros(Q.shape), np.zeros(Q.shape)
        for b in range(3):
            for t in range(cu[b], cu[b + 1]):
                ref[t:t + 1], size[t:t + 1] = layer.kv_attention(Q[t:t + 1], kc, ks, vc, vs, table[b:b + 1], [lens[b]], [0, 1], 0.4)
    assert np.allclose(O, ref) and np.allclose(A, size)


def test_gated_gradient_against_differences():
    g = np.random.default_rng(3)
    I = 24
    GU = 2 * g.standard_normal((3, 2 * I))
    A, sA = oq.quant_1x128(g.standard_normal((3, 16)).astype(np.float32), fmt="e5m2")
    W, sW = oq.quant_128x128(g.standard_normal((I, 16)).astype(np.float32))
    dg, du, dh = layer.gated_backward(A, sA, W, sW, GU)
    d = 1e-5
    f = lambda gu: dh * (gu[:, :I] / (1 + np.exp(-gu[:, :I])) * gu[:, I:])  # noqa: E731
    one = np.concatenate((np.full(I, d), np.zeros(I)))
    two = np.concatenate((np.zeros(I), np.full(I, d)))
    assert np.allclose((f(GU + one) - f(GU - one)) / (2 * d), dg, atol=1e-7)
    assert np.allclose((f(GU + two) - f(GU - two)) / (2 * d), du, atol=1e-7)


def test_gated_is_the_products_and_silu():
    g = np.random.default_rng(4)
    A, sA = oq.quant_1x128(g.standard_normal((4, 160)).astype(np.float32))
    W, sW = oq.quant_128x128(g.standard_normal((96, 160)).astype(np.float32))
    h, u = layer.gated(A, sA, W, sW)
    x = layer.e4m3.decode(A) * np.repeat(sA, 128, 1)[:, :160]
    w = layer.e4m3.decode(W) * np.repeat(sW, 128, 1)[:, :160]
    assert np.allclose(u, x @ w.T, rtol=1e-6) and np.allclose(h, u[:, :48] / (1 + np.exp(-u[:, :48])) * u[:, 48:])
