"""fp8gemm_gated and fp8gemm_gated_backward against the FP64 oracle.

Bounds, derived before the first run.  S is the sum of the magnitudes of a product's terms.
  products  FP8 products are exact; 128 of them are summed in FP32 on the tensor cores (32 at a
            time: at most 40 roundings of 2^-23), then K / 128 promoted in FP32:
            e = (K / 128 + 40) 2^-23 S
  h         silu has slope 1.1 at most; exponential, quotient and products 2^-20:
            eh = 1.1 |u| e_g + |silu(g)| e_u + 2^-20 |h|
  gradients dg = dh u s (1 + g (1 - s)): factors from FP32 of exact inputs, the bracket within
            2^-21 (1 + |g|) of terms, the rest relative 2^-20:
            e_dg = |u s| (|1 + g (1 - s)| e + |dh| 2^-20 (1 + |g|)),  e_du = |g s| (e + 2^-20 |dh|)
  scales    within max e / limit and 2^-22 of the oracle's
  codes     between those of the two ends of (value -+ e) / scale, each widened by 2^-22
  BF16      e and half a step (2^-8)
"""

import numpy as np
import pytest

from oracle import layer
from oracle import quant as oq
from tests.gpu_helpers import dev, host

pytestmark = pytest.mark.gpu

_CODES = {"e4m3": layer.e4m3, "e5m2": layer.e5m2}
_LIMIT = {"e4m3": 448.0, "e5m2": 57344.0}


def _operands(M, N, K, fmt, seed, spread=3):
    g = np.random.default_rng(seed)
    X = (g.standard_normal((M, K)) * np.exp2(spread * g.standard_normal((M, 1)))).astype(np.float32)
    W = (g.standard_normal((N, K)) / np.sqrt(K) * np.exp2(g.integers(-1, 2, (N, 1)))).astype(np.float32)
    return (*oq.quant_1x128(X, fmt=fmt), *oq.quant_128x128(W))


def _sizes(A, sA, W, sW, fmt):
    a = np.abs(_CODES[fmt].decode(A)) * np.repeat(sA.astype(np.float64), 128, 1)[:, :A.shape[1]]
    K = A.shape[1]
    return (-(-K // 128) + 40) * 2.0 ** -23 * (a @ np.abs(layer._dequant(W, sW)).T)


def _check_codes(Q, sQ, ref, err, fmt):
    """1x128 codes and scales of ref known to err."""
    codes, limit = _CODES[fmt], _LIMIT[fmt]
    s = sQ.astype(np.float64)
    assert s.shape == (ref.shape[0], -(-ref.shape[1] // 128))
    for kb in range(s.shape[1]):
        r, e = (x[:, 128 * kb:128 * kb + 128] for x in (ref, err))
        sr = np.max(np.abs(r), axis=1) / limit
        assert np.all(np.abs(s[:, kb] - sr) <= np.max(e, axis=1) / limit + 2.0 ** -22 * sr)
        z = np.where(s[:, kb] > 0, s[:, kb], 1)[:, None]
        low, high = (r - e) / z, (r + e) / z
        low, high = low - np.abs(low) * 2.0 ** -22, high + np.abs(high) * 2.0 ** -22
        a, b = (codes.decode(codes.encode_rne_sat(x.astype(np.float32))) for x in (low, high))
        v = codes.decode(Q[:, 128 * kb:128 * kb + 128])
        assert np.all((v >= a) & (v <= b))


def _check_bf16(got, ref, err):
    assert np.all(np.abs(host(got) - ref) <= err * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref))


SHAPES = [(1, 16, 16), (1, 7168, 128), (3, 400, 400), (64, 1040, 272), (65, 4096, 48), (130, 272, 144), (200, 2064, 112),
          (300, 512, 1040), (129, 2048, 2064), (1300, 144, 2048), (2500, 256, 1296),
          (2700, 144, 2064), (2700, 16, 2064)]  # the last two: several tiles a CTA


@pytest.mark.parametrize("M,K,I", SHAPES)
@pytest.mark.parametrize("a_fmt,fmt,save", [("e4m3", "e4m3", True), ("e5m2", "e4m3", False), ("e4m3", "e5m2", True)])
def test_forward(M, K, I, a_fmt, fmt, save):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    A, sA, W, sW = _operands(M, 2 * I, K, a_fmt, seed=M + K + I, spread=1)
    GU = torch.full((M, 2 * I), float("nan"), dtype=torch.bfloat16, device="cuda") if save else None
    Q, sQ = b.fp8gemm_gated(dev(A), dev(sA), dev(W), dev(sW), a_fmt=a_fmt, fmt=fmt, GU=GU)
    h, u = layer.gated(A, sA, W, sW, a_fmt)
    e = _sizes(A, sA, W, sW, a_fmt)
    g, up = u[:, :I], u[:, I:]
    eh = 1.1 * np.abs(up) * e[:, :I] + np.abs(g / (1 + np.exp(-g))) * e[:, I:] + 2.0 ** -20 * np.abs(h)
    _check_codes(host(Q), host(sQ), h, eh, fmt)
    if save:
        _check_bf16(GU, u, e)
        Q2, sQ2 = b.fp8gemm_gated(dev(A), dev(sA), dev(W), dev(sW), a_fmt=a_fmt, fmt=fmt)
        assert torch.equal(Q, Q2) and torch.equal(sQ, sQ2)
    assert b.fp8gemm_get_device_status() == b.OK


@pytest.mark.parametrize("M,K,I", SHAPES)
@pytest.mark.parametrize("a_fmt,fmt,save", [("e5m2", "e5m2", True), ("e4m3", "e4m3", False)])
def test_backward(M, K, I, a_fmt, fmt, save):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    A, sA, W, sW = _operands(M, I, K, a_fmt, seed=M + K + I)
    r = np.random.default_rng(I)
    tGU = dev((3 * r.standard_normal((M, 2 * I))).astype(np.float32)).to(torch.bfloat16)
    GU = tGU.double().cpu().numpy()
    dGU = torch.full((M, 2 * I), float("nan"), dtype=torch.bfloat16, device="cuda") if save else None
    Ip = 128 * (-(-I // 128))
    Q = torch.full((M, 2 * Ip), 0x55, dtype=torch.uint8, device="cuda")
    _, sQ = b.fp8gemm_gated_backward(dev(A), dev(sA), dev(W), dev(sW), tGU, a_fmt=a_fmt, fmt=fmt, dGU=dGU, Q=Q)
    dg, du, dh = layer.gated_backward(A, sA, W, sW, GU, a_fmt)
    e = _sizes(A, sA, W, sW, a_fmt)
    g, u = GU[:, :I], GU[:, I:]
    s = 1 / (1 + np.exp(-g))
    eg = np.abs(u * s) * (np.abs(1 + g * (1 - s)) * e + np.abs(dh) * 2.0 ** -20 * (1 + np.abs(g)))
    eu = np.abs(g * s) * (e + 2.0 ** -20 * np.abs(dh))
    Qh, sh = host(Q), host(sQ)
    for i, (x, ex) in enumerate(((dg, eg), (du, eu))):
        _check_codes(Qh[:, i * Ip:i * Ip + I], sh[:, i * (Ip // 128):(i + 1) * (Ip // 128)], x, ex, fmt)
        assert not Qh[:, i * Ip + I:(i + 1) * Ip].any()
    if save:
        _check_bf16(dGU, np.concatenate((dg, du), 1), np.concatenate((eg, eu), 1))
    assert b.fp8gemm_get_device_status() == b.OK


def test_gradient_against_differences():
    """dGU against central differences in FP64 of sum(dh silu(g) u), dh the product's own value: third derivatives
    of silu are below 1, so a step of 2^-10 is off by 2^-21 |dh u| and rounds to 2^-40."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    M, K, I = 70, 256, 160
    A, sA, W, sW = _operands(M, I, K, "e5m2", seed=5)
    r = np.random.default_rng(6)
    tGU = dev((4 * r.standard_normal((M, 2 * I))).astype(np.float32)).to(torch.bfloat16)
    dGU = torch.empty((M, 2 * I), dtype=torch.bfloat16, device="cuda")
    b.fp8gemm_gated_backward(dev(A), dev(sA), dev(W), dev(sW), tGU, dGU=dGU)
    GU = tGU.double().cpu().numpy()
    g, u = GU[:, :I], GU[:, I:]
    x = layer._FORMATS["e5m2"][2](A) * np.repeat(sA.astype(np.float64), 128, 1)
    dh = x @ layer._dequant(W, sW).T
    e = _sizes(A, sA, W, sW, "e5m2")
    silu = lambda t: t / (1 + np.exp(-t))  # noqa: E731
    d = 2.0 ** -10
    dg, du = dh * u * (silu(g + d) - silu(g - d)) / (2 * d), dh * silu(g) * ((u + d) - (u - d)) / (2 * d)
    eg = 1.1 * np.abs(u) * (e + np.abs(dh) * (2.0 ** -20 * (1 + np.abs(g)) + 2.0 ** -20))
    eu = np.abs(silu(g)) * (e + 2.0 ** -20 * np.abs(dh))
    _check_bf16(dGU, np.concatenate((dg, du), 1), np.concatenate((eg, eu), 1))


@pytest.mark.parametrize("gate", [-1e4, -80.0, 80.0, 1e4])
def test_saturated_gates(gate):
    """Gates where the sigmoid is 0 or 1 (and e^-g infinite): values and gradients stay finite and right."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    M, I = 5, 144
    GU = torch.full((M, 2 * I), gate, dtype=torch.bfloat16, device="cuda")
    GU[:, I:] = 2.0
    A, W = torch.full((M, 16), 0x38, dtype=torch.uint8, device="cuda"), torch.full((I, 16), 0x38, dtype=torch.uint8, device="cuda")
    one = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    dGU = torch.empty_like(GU)
    b.fp8gemm_gated_backward(A, one(M, 1), W, one(2, 1), GU, a_fmt="e4m3", dGU=dGU)
    g = float(GU[0, 0])
    s = 1 / (1 + np.exp(-np.float64(g))) if g > -700 else 0.0
    want = 16 * 2 * s * (1 + g * (1 - s)), 16 * g * s
    for got, w in ((dGU[:, :I], want[0]), (dGU[:, I:], want[1])):
        got = host(got)
        assert np.all(np.abs(got - w) <= 2.0 ** -8 * abs(w) + 1e-30)
    W1 = torch.full((2 * I, 16), 0x38, dtype=torch.uint8, device="cuda")
    s1 = one(3, 1)
    sA = one(M, 1) * (gate / 16)  # u = gate in every column
    Q, sQ = b.fp8gemm_gated(A, sA, W1, s1)
    h = (torch.sign(torch.tensor(gate)) > 0) * float(gate) ** 2
    got = Q.view(torch.float8_e4m3fn).float() * sQ.repeat_interleave(128, 1)[:, :I]
    assert bool(((got - float(h)).abs() <= 2.0 ** -4 * float(h) + 1e-30).all())


@pytest.mark.parametrize("M,I", [(5, 144), (2700, 2064)])
@pytest.mark.parametrize("gate,up", [(-1e30, 1e10), (-3e38, -3e38), (1e30, 1e7), (-1e20, 3e38)])
def test_gates_and_up_values_whose_product_leaves_fp32(M, I, gate, up):
    """The sigmoid's 0 takes the gradients with it, its 1 leaves dh u and dh g, whatever the product of gate and up value
    (dh = 2^-20 times 16 products of ones: exact)."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    GU = torch.full((M, 2 * I), gate, dtype=torch.bfloat16, device="cuda")
    GU[:, I:] = up
    A, W = torch.full((M, 16), 0x38, dtype=torch.uint8, device="cuda"), torch.full((I, 16), 0x38, dtype=torch.uint8, device="cuda")
    dGU = torch.empty_like(GU)
    Q, sQ = b.fp8gemm_gated_backward(A, torch.full((M, 1), 2.0 ** -20, device="cuda"), W, torch.ones((-(-I // 128), 1), device="cuda"),
                                     GU, a_fmt="e4m3", dGU=dGU)
    want = torch.zeros_like(GU) if gate < 0 else torch.cat((GU[:, I:], GU[:, :I]), 1) * 2.0 ** -16
    assert torch.equal(dGU, want)
    if gate < 0:
        assert not bool(sQ.any()) and not bool(Q.any())


def test_rows_of_zeros_and_nan():
    """A row of zeros has scale 0 and zero codes; a NaN scale makes its row's scales NaN, no other's."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    A, sA, W, sW = _operands(200, 544, 256, "e4m3", seed=9, spread=1)
    A[7] = 0
    sA[9, 1] = np.nan
    Q, sQ = b.fp8gemm_gated(dev(A), dev(sA), dev(W), dev(sW))
    q, s = host(Q), host(sQ)
    assert not q[7].any() and not s[7].any()
    assert np.isnan(s[9]).all() and np.isfinite(np.delete(s, 9, 0)).all()


def test_same_bits_on_every_run_and_in_a_graph():
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    for M, K, I in ((3, 2048, 272), (700, 512, 1040)):
        A, sA, W, sW = (dev(x) for x in _operands(M, 2 * I, K, "e4m3", seed=M))
        want = b.fp8gemm_gated(A, sA, W, sW)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                got = b.fp8gemm_gated(A, sA, W, sW)
            for _ in range(3):
                got[0].zero_()
                graph.replay()
                s.synchronize()
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert b.fp8gemm_get_device_status() == b.OK


def test_no_rows():
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    f = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    Q, sQ = b.fp8gemm_gated(z(0, 256), f(0, 2), z(64, 256), f(1, 2))
    assert Q.shape == (0, 32) and sQ.shape == (0, 1)
    Q, sQ = b.fp8gemm_gated_backward(z(0, 256), f(0, 2), z(32, 256), f(1, 2),
                                     torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    assert Q.shape == (0, 256)
