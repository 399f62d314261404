"""The FP64 statements of the decoder layer's operators against closed forms,
differences and library routines.  CPU only."""

import numpy as np
import pytest
import torch

from oracle import e4m3, layer, quant


def test_norm_closed_forms():
    X = np.array([[3.0, -4.0] * 8])
    h, rstd, y = layer.rmsnorm(X, None, np.full(16, 2.0), 0.0, True)
    assert rstd[0] == pytest.approx(1 / np.sqrt(12.5), rel=1e-15)
    assert np.allclose(y, X * 2 / np.sqrt(12.5), rtol=1e-15)
    h, _, _ = layer.rmsnorm(X, np.full((1, 16), 1 / 512), np.ones(16), 0.0, True)
    assert np.array_equal(h, [[3.0, -4.0] * 8])  # the sum is rounded to BF16
    _, rstd, y = layer.rmsnorm(np.zeros((1, 16)), None, np.ones(16), 1e-6, True)
    assert rstd[0] == pytest.approx(1e3) and not y.any()


def test_norm_gradient_against_differences():
    g = np.random.default_rng(0)
    M, K, eps, d = 3, 32, 1e-3, 1e-5
    X, gain, dY, dH = (g.standard_normal(s) for s in ((M, K), K, (M, K), (M, K)))

    def loss(x, w):
        _, _, y = layer.rmsnorm(x, None, w, eps, False)
        return np.sum(y * dY) + np.sum(x * dH)

    h, rstd, _ = layer.rmsnorm(X, None, gain, eps, False)
    dX, dG = layer.rmsnorm_backward(dY, h, rstd, gain, dH)
    for m, k in [(0, 0), (1, 7), (2, 31)]:
        e = np.zeros((M, K))
        e[m, k] = d
        assert (loss(X + e, gain) - loss(X - e, gain)) / (2 * d) == pytest.approx(dX[m, k], rel=1e-7, abs=1e-8)
    for k in (0, 5, 31):
        e = np.zeros(K)
        e[k] = d
        assert (loss(X, gain + e) - loss(X, gain - e)) / (2 * d) == pytest.approx(dG[k], rel=1e-7, abs=1e-8)


def test_pow2_scale():
    assert layer.pow2_scale(448.0, 448.0) == 1.0
    assert layer.pow2_scale(450.0, 448.0) == 2.0
    assert layer.pow2_scale(224.0, 448.0) == 0.5
    assert layer.pow2_scale(0.0, 448.0) == 0.0
    assert layer.pow2_scale(1e-40, 448.0) == 2.0 ** -126


def test_append_grows_a_scale_and_keeps_values():
    cache = np.zeros((3, 1, 16, 64), np.uint8)
    scale = np.full((3, 1), 7.0, np.float32)  # stale: a fresh block ignores it
    table = np.array([[2, 0]])
    a = np.full((3, 1, 64), 0.5, np.float32)
    layer.kv_append(a, cache, scale, table, [3], [0, 3])
    s0 = scale[2, 0]
    assert s0 == 2.0 ** -9 and np.all(e4m3.decode(cache[2, 0, :3]) * s0 == 0.5)
    layer.kv_append(np.full((1, 1, 64), 100.0, np.float32), cache, scale, table, [4], [0, 1])
    assert scale[2, 0] == 0.25 and np.all(e4m3.decode(cache[2, 0, :3]) * 0.25 == 0.5)
    layer.kv_append(np.zeros((14, 1, 64), np.float32), cache, scale, table, [18], [0, 14])
    assert scale[2, 0] == 0.25 and scale[0, 0] == 0.0 and scale[1, 0] == 7.0


def test_attention_against_a_library_softmax():
    g = np.random.default_rng(1)
    kc = e4m3.encode_rne_sat(g.standard_normal((4, 2, 16, 64)).astype(np.float32))
    vc = e4m3.encode_rne_sat(g.standard_normal((4, 2, 16, 64)).astype(np.float32))
    ks, vs = np.full((4, 2), 0.5, np.float32), np.full((4, 2), 2.0, np.float32)
    Q = g.standard_normal((2, 4, 64))
    O, _ = layer.kv_attention(Q, kc, ks, vc, vs, np.array([[3, 1]]), [20], [0, 2], 0.125)
    k = torch.from_numpy(np.concatenate([e4m3.decode(kc[3]), e4m3.decode(kc[1])], 1)[:, :20] * 0.5)
    v = torch.from_numpy(np.concatenate([e4m3.decode(vc[3]), e4m3.decode(vc[1])], 1)[:, :20] * 2.0)
    q = torch.from_numpy(Q).transpose(0, 1)
    mask = torch.tensor([[True] * 19 + [False], [True] * 20])
    ref = torch.nn.functional.scaled_dot_product_attention(
        q, k.repeat_interleave(2, 0), v.repeat_interleave(2, 0), attn_mask=mask, scale=0.125)
    assert np.allclose(O, ref.transpose(0, 1).numpy(), rtol=1e-12, atol=1e-12)
    # more queries than cached tokens: the first sees nothing
    O, _ = layer.kv_attention(Q, kc, ks, vc, vs, np.array([[3, 1]]), [1], [0, 2], 0.125)
    assert not O[0].any() and np.allclose(O[1], np.repeat(v[:, 0].numpy(), 2, 0))


def test_route():
    ids, w = layer.moe_route([[1.0, 3.0, 3.0, -np.inf, 2.0]], 4)
    assert ids.tolist() == [[1, 2, 4, 0]]
    ref = torch.softmax(torch.tensor([3.0, 3.0, 2.0, 1.0], dtype=torch.float64), 0).numpy()
    assert np.allclose(w, ref)
    _, w = layer.moe_route([[1.0, 3.0, 3.0, -np.inf, 2.0]], 1, renormalise=False)
    assert w[0, 0] == pytest.approx(np.exp(3) / (np.exp(1) + 2 * np.exp(3) + np.exp(2)))


def test_moe_of_one_expert_is_the_dense_chain():
    g = np.random.default_rng(2)
    T, H, I = 2, 144, 160
    A, sA = quant.quant_1x128(g.standard_normal((T, H)).astype(np.float32))
    W1, s1 = quant.quant_128x128(g.standard_normal((2 * I, H)).astype(np.float32))
    W2, s2 = quant.quant_128x128(g.standard_normal((H, I)).astype(np.float32))
    out, _, w = layer.moe(A, sA, np.zeros((T, 1)), W1[None], s1[None], W2[None], s2[None], 1)
    assert np.all(w == 1)
    from oracle import gemm
    u = gemm.gemm_dense(A, sA, W1, s1)
    h = u[:, :I] / (1 + np.exp(-u[:, :I])) * u[:, I:]
    h8, sh = quant.quant_1x128(h.astype(np.float32))
    ref = gemm.gemm_dense(h8, sh, W2, s2)
    assert np.linalg.norm(out - ref) < 1e-5 * np.linalg.norm(ref)
