"""fp8_rmsnorm_quant and fp8_rmsnorm_backward against the FP64 oracle.

Bounds, derived before the first run (u = 2^-24, FP32 rounding):
  rstd   a sum of squares in at most 16 + 11 levels of additions, a division, a
         sum, a root: under 32 u = 2e-6 relative
  y      rstd and two products: 2.2e-6 relative; the block's scale adds a
         division: 2.5e-6
  codes  are those of some y / s within 5e-6 relative of the oracle's: between
         the codes of the two ends
  dx     sums and products of FP32: 2^-18 of the sum of its terms' magnitudes,
         and half a BF16 step (2^-9) of the result
  dg     at most 8192 / 152 + 16 additions in sequence and the terms' own
         rounding: 2^-17 of the sum of magnitudes
"""

import numpy as np
import pytest

from oracle import layer
from tests.gpu_helpers import dev, host

pytestmark = pytest.mark.gpu

_CODES = {"e4m3": layer.e4m3, "e5m2": layer.e5m2}
EPS = 1e-6


def _inputs(M, K, kind, residual, seed):
    import torch
    g = np.random.default_rng(seed)
    t = torch.bfloat16 if kind == "bf16" else torch.float32
    X = g.standard_normal((M, K)).astype(np.float32)
    X[:, ::37] *= 40
    if M > 2:
        X[1] = 0
        X[2] *= 1e-18
    R = (2 * g.standard_normal((M, K))).astype(np.float32) if residual else None
    if R is not None and M > 2:
        R[1] = 0
    gain = (1 + 0.2 * g.standard_normal(K)).astype(np.float32)
    if K >= 256:
        gain[128:256] = 0  # a block of zeros in every row
    tX = dev(X).to(t)
    tR = dev(R).to(t) if residual else None
    return tX, tR, dev(gain), tX.double().cpu().numpy(), (tR.double().cpu().numpy() if residual else None), gain


def _check_forward(got, X, R, gain, kind, fmt):
    Q, sQ, H, rstd = got
    h, r, y = layer.rmsnorm(X, R, gain, EPS, kind == "bf16")
    assert np.array_equal(H.double().cpu().numpy(), h)
    assert np.all(np.abs(host(rstd) - r) <= 2e-6 * r)
    codes = _CODES[fmt]
    limit = 448.0 if fmt == "e4m3" else 57344.0
    M, K = y.shape
    q, s = host(Q.view(M, K)), host(sQ).reshape(M, -1).astype(np.float64)
    for kb in range(s.shape[1]):
        yb = y[:, 128 * kb:128 * kb + 128]
        sr = np.max(np.abs(yb), axis=1) / limit
        tiny = sr < 2.0 ** -126  # a subnormal scale: no relative bound
        assert np.all((np.abs(s[:, kb] - sr) <= 2.5e-6 * sr) | tiny)
        z = yb[~tiny] / np.where(sr > 0, sr, 1)[~tiny, None]
        a = codes.decode(codes.encode_rne_sat((z * (1 - 5e-6)).astype(np.float32)))
        b = codes.decode(codes.encode_rne_sat((z * (1 + 5e-6)).astype(np.float32)))
        v = codes.decode(q[:, 128 * kb:128 * kb + 128][~tiny])
        assert np.all((v >= np.minimum(a, b)) & (v <= np.maximum(a, b)))


@pytest.mark.parametrize("M,K,kind,fmt,residual", [
    (1, 16, "bf16", "e4m3", True), (3, 144, "f32", "e4m3", False), (5, 400, "bf16", "e5m2", True),
    (7, 2064, "f32", "e5m2", True), (64, 2048, "bf16", "e4m3", False), (1, 7168, "bf16", "e4m3", True),
    (33, 7168, "bf16", "e4m3", True), (3, 8208, "bf16", "e4m3", True), (2, 16384, "f32", "e4m3", True),
    (700, 256, "bf16", "e4m3", True), (2000, 528, "f32", "e4m3", True)])
def test_forward(M, K, kind, fmt, residual):
    from fp8_fine_grained_e4m3_gb300 import binding as b
    tX, tR, tg, X, R, gain = _inputs(M, K, kind, residual, seed=M + K)
    got = b.fp8_rmsnorm_quant(tX, tg, EPS, residual=tR, fmt=fmt)
    if not residual:
        assert got[2] is tX
    _check_forward(got, X, R, gain, kind, fmt)
    again = b.fp8_rmsnorm_quant(tX, tg, EPS, residual=tR, fmt=fmt)
    for x, y in zip(got, again):
        assert bool((x == y).all())


def test_forward_updates_the_stream_in_place_on_another_stream():
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    tX, tR, tg, X, R, gain = _inputs(40, 1040, "bf16", True, seed=3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = b.fp8_rmsnorm_quant(tX, tg, EPS, residual=tR, H=tR, stream=s)
    s.synchronize()
    assert got[2] is tR
    _check_forward(got, X, R, gain, "bf16", "e4m3")


def test_forward_feeds_the_gemm_without_host_sync():
    """norm -> GEMM -> norm chained on one stream equals the calls one by one."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = np.random.default_rng(5)
    B, sB = b.fp8_quant_128x128(dev((0.05 * g.standard_normal((1024, 1024))).astype(np.float32)))
    for M in (1, 48, 300):
        x = dev(g.standard_normal((M, 1024)).astype(np.float32)).to(torch.bfloat16)
        gain = dev(np.ones(1024, np.float32))
        outs = []
        for sync in (False, True):
            h, y = x, x
            for _ in range(3):
                Q, sQ, h, _ = b.fp8_rmsnorm_quant(y, gain, EPS, residual=h)
                if sync:
                    torch.cuda.synchronize()
                y = b.fp8gemm_dense(Q, sQ, B, sB)
                if sync:
                    torch.cuda.synchronize()
            outs.append((h, y))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("M,K,kind,residual", [
    (1, 16, "f32", True), (3, 144, "bf16", True), (130, 400, "f32", False), (65, 2064, "bf16", True),
    (9, 7168, "f32", True), (700, 1024, "bf16", False), (4, 8208, "bf16", True), (3, 16384, "f32", True),
    (8192, 128, "bf16", True)])
def test_backward(M, K, kind, residual):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    tX, _, tg, X, _, gain = _inputs(M, K, kind, False, seed=M * K)
    g = np.random.default_rng(M)
    tdY = dev((0.1 * g.standard_normal((M, K))).astype(np.float32)).to(tX.dtype)
    tdH = dev(g.standard_normal((M, K)).astype(np.float32)).to(tX.dtype) if residual else None
    _, _, _, rstd = b.fp8_rmsnorm_quant(tX, tg, EPS)
    dX, dG = b.fp8_rmsnorm_backward(tdY, tX, rstd, tg, dH=tdH)
    dY, dH = tdY.double().cpu().numpy(), (tdH.double().cpu().numpy() if residual else None)
    rx, rg = layer.rmsnorm_backward(dY, X, host(rstd), gain, dH)
    r = host(rstd).astype(np.float64)[:, None]
    terms = np.abs(r * dY * gain) + np.abs(X * r * r) * np.mean(np.abs(dY * gain * X * r), 1, keepdims=True)
    if residual:
        terms = terms + np.abs(dH)
    bound = 2.0 ** -18 * terms + (2.0 ** -8 * np.abs(rx) if kind == "bf16" else 0)
    assert np.all(np.abs(dX.double().cpu().numpy() - rx) <= bound)
    assert np.all(np.abs(host(dG) - rg) <= 2.0 ** -17 * np.sum(np.abs(dY * X * r), 0))
    dX2, dG2 = b.fp8_rmsnorm_backward(tdY, tX, rstd, tg, dH=tdH)
    assert torch.equal(dX, dX2) and torch.equal(dG, dG2)
    if residual:  # in place on the stream's gradient
        b.fp8_rmsnorm_backward(tdY, tX, rstd, tg, dH=tdH, dX=tdH)
        assert torch.equal(tdH, dX)


def test_backward_against_differences():
    """The FP32 gradient against differences of the FP64 norm."""
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = np.random.default_rng(8)
    M, K, d = 2, 144, 1e-4
    X, dY = g.standard_normal((M, K)).astype(np.float32), g.standard_normal((M, K)).astype(np.float32)
    gain = g.standard_normal(K).astype(np.float32)
    _, _, _, rstd = b.fp8_rmsnorm_quant(dev(X), dev(gain), EPS)
    dX, dG = (host(t) for t in b.fp8_rmsnorm_backward(dev(dY), dev(X), rstd, dev(gain)))

    def loss(x, w):
        return np.sum(layer.rmsnorm(x, None, w, EPS, False)[2] * dY.astype(np.float64))

    for m, k in [(0, 0), (0, 143), (1, 77)]:
        e = np.zeros((M, K))
        e[m, k] = d
        diff = (loss(X + e, gain) - loss(X - e, gain)) / (2 * d)
        assert abs(diff - dX[m, k]) < 1e-4
    for k in (0, 99):
        e = np.zeros(K)
        e[k] = d
        assert abs((loss(X, gain + e) - loss(X, gain - e)) / (2 * d) - dG[k]) < 1e-4


def test_no_rows():
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    gain = torch.ones(256, device="cuda")
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    Q, sQ, _, rstd = b.fp8_rmsnorm_quant(x, gain)
    assert Q.shape == (0, 256) and sQ.shape == (0, 2) and rstd.shape == (0,)
    dG = torch.full((256,), 3.0, device="cuda")
    b.fp8_rmsnorm_backward(x, x, rstd, gain, dgain=dG)
    assert not dG.any()


@pytest.mark.parametrize("M,K,kind,residual", [(3, 400, "bf16", True), (5, 7168, "f32", False), (320, 2048, "bf16", True),
                                               (310, 7168, "f32", True), (2, 16384, "bf16", False)])
@pytest.mark.parametrize("size,eps", [(1e25, EPS), (1e38, 0.0), (1e-30, 0.0), (3e-21, 0.0), (1e-18, 1e-36)])
def test_squares_past_the_range_of_fp32(M, K, kind, residual, size, eps):
    """Finite rows whose squares over- or underflow, beside an ordinary row and one
    of zeros.  Bounds as above: the sum is the same one, of h times a power of two."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = np.random.default_rng(K)
    t = torch.bfloat16 if kind == "bf16" else torch.float32
    X, R = (g.uniform(0.25, 1, (M, K)).astype(np.float32) * np.float32(size) for _ in range(2))
    X[0], R[0] = g.standard_normal(K), g.standard_normal(K)
    X[-1] = R[-1] = 0
    gain = (1 + 0.2 * g.standard_normal(K)).astype(np.float32)
    tX, tR = dev(X).to(t), dev(R).to(t) if residual else None
    got = b.fp8_rmsnorm_quant(tX, dev(gain), eps, residual=tR)
    live = slice(0, M - 1)
    h, r, y = layer.rmsnorm(tX.double().cpu().numpy()[live], tR.double().cpu().numpy()[live] if residual else None, gain,
                            eps, kind == "bf16")
    assert np.array_equal(got[2].double().cpu().numpy()[live], h)
    assert np.all(np.abs(host(got[3])[live] - r) <= 2e-6 * r)
    q, s = host(got[0]), host(got[1]).astype(np.float64)
    amax = np.stack([np.max(np.abs(y[:, k:k + 128]), 1) for k in range(0, K, 128)], 1)
    assert np.all(np.abs(s[live] - amax / 448) <= 2.5e-6 * amax / 448)
    v = layer.e4m3.decode(q[live]) * np.repeat(s[live], 128, 1)[:, :K]
    assert np.all(np.abs(v - y) <= np.abs(y) / 15 + np.repeat(amax / 448, 128, 1)[:, :K] * 2.0 ** -9)
    assert not q[-1].any() and not s[-1].any()


@pytest.mark.parametrize("K,M,kind", [(400, 3, "bf16"), (7168, 2, "f32"), (2048, 320, "bf16")])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_a_row_that_is_not_finite_stays_so(K, M, kind, bad, fmt):
    """One NaN or infinity: the row's product with anything is NaN, other rows are
    what they were."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = np.random.default_rng(4)
    X = g.standard_normal((M, K)).astype(np.float32)
    t = torch.bfloat16 if kind == "bf16" else torch.float32
    gain = dev((1 + 0.2 * g.standard_normal(K)).astype(np.float32))
    clean = b.fp8_rmsnorm_quant(dev(X).to(t), gain, EPS, fmt=fmt)
    X[1, K - 3] = bad
    got = b.fp8_rmsnorm_quant(dev(X).to(t), gain, EPS, fmt=fmt)
    values = _CODES[fmt].decode(host(got[0])) * np.repeat(host(got[1]), 128, 1)[:, :K]
    rows = np.arange(M) != 1
    assert np.isnan(values[1].sum())
    assert np.isfinite(values[rows]).all()
    for a, c in zip(got[:2], clean[:2]):
        assert np.array_equal(host(a)[rows], host(c)[rows])
    if np.isnan(bad):
        assert np.isnan(host(got[1])[1]).all()
    W, sW = b.fp8_quant_128x128(dev(g.standard_normal((128, K)).astype(np.float32)))
    D = b.fp8gemm_dense_fmt(got[0], got[1], fmt, W, sW, "e4m3")
    assert bool(D[1].isnan().all()) and bool(D[torch.from_numpy(rows).cuda()].isfinite().all())


def test_a_gain_that_is_not_a_number_shows():
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = np.random.default_rng(5)
    X, gain = g.standard_normal((2, 512)).astype(np.float32), np.ones(512, np.float32)
    gain[128:256] = np.nan
    _, s, _, _ = b.fp8_rmsnorm_quant(dev(X), dev(gain), EPS)
    assert np.array_equal(np.isnan(host(s)), [[False, True, False, False]] * 2)


def test_a_scale_that_underflows():
    """|y| of at most 2e-43 in a block: its scale is 0 in FP32, its codes are zeros,
    and the row's product is that of the other blocks."""
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = np.random.default_rng(6)
    X, gain = g.uniform(-1, 1, (3, 384)).astype(np.float32), np.ones(384, np.float32)
    X[:, ::5] = 0
    gain[128:256] = 1e-43
    Q, s, _, _ = b.fp8_rmsnorm_quant(dev(X), dev(gain), EPS)
    assert not host(Q)[:, 128:256].any() and not host(s)[:, 1].any()
    assert host(Q)[:, :128].any() and host(s)[:, 0].all()
    W, sW = b.fp8_quant_128x128(dev(g.standard_normal((128, 384)).astype(np.float32)))
    assert bool(b.fp8gemm_dense(Q, s, W, sW).isfinite().all())


@pytest.mark.parametrize("M,K,kind,fmt,residual", [
    (400, 2048, "bf16", "e4m3", True), (320, 7168, "bf16", "e5m2", True), (310, 16384, "f32", "e4m3", False),
    (305, 8208, "f32", "e4m3", True), (330, 7168, "bf16", "e4m3", False)])
def test_forward_of_rows_in_four_chunks_a_thread(M, K, kind, fmt, residual):
    """Rows for every SM and wide: the form that a prompt takes.  Its sum of squares is 32
    terms in sequence in a thread, then 5 + 4 levels of additions, a division and a sum:
    at most 43 u of itself, so rstd at most 21.5 u + 1 u = 1.4e-6: within the 2e-6 above."""
    from fp8_fine_grained_e4m3_gb300 import binding as b
    tX, tR, tg, X, R, gain = _inputs(M, K, kind, residual, seed=M + K)
    _check_forward(b.fp8_rmsnorm_quant(tX, tg, EPS, residual=tR, fmt=fmt), X, R, gain, kind, fmt)


@pytest.mark.parametrize("M,K,kind,residual", [
    (1300, 4096, "bf16", True), (400, 16384, "f32", True), (500, 8208, "bf16", False), (1400, 2048, "f32", True),
    (2000, 1024, "bf16", True)])
def test_backward_of_ctas_that_take_several_rows(M, K, kind, residual):
    """CTAs of several warps with more than one row each, in all three shapes.  dg: at
    most 14 rows in sequence in a thread and 10 + 5 partials: below the 2^-17 above."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    tX, _, tg, X, _, gain = _inputs(M, K, kind, False, seed=M * K)
    g = np.random.default_rng(M)
    tdY = dev((0.1 * g.standard_normal((M, K))).astype(np.float32)).to(tX.dtype)
    tdH = dev(g.standard_normal((M, K)).astype(np.float32)).to(tX.dtype) if residual else None
    _, _, _, rstd = b.fp8_rmsnorm_quant(tX, tg, EPS)
    dX, dG = b.fp8_rmsnorm_backward(tdY, tX, rstd, tg, dH=tdH)
    dY, dH = tdY.double().cpu().numpy(), (tdH.double().cpu().numpy() if residual else None)
    rx, rg = layer.rmsnorm_backward(dY, X, host(rstd), gain, dH)
    r = host(rstd).astype(np.float64)[:, None]
    terms = np.abs(r * dY * gain) + np.abs(X * r * r) * np.mean(np.abs(dY * gain * X * r), 1, keepdims=True)
    if residual:
        terms = terms + np.abs(dH)
    bound = 2.0 ** -18 * terms + (2.0 ** -8 * np.abs(rx) if kind == "bf16" else 0)
    assert np.all(np.abs(dX.double().cpu().numpy() - rx) <= bound)
    assert np.all(np.abs(host(dG) - rg) <= 2.0 ** -17 * np.sum(np.abs(dY * X * r), 0))
    dX2, dG2 = b.fp8_rmsnorm_backward(tdY, tX, rstd, tg, dH=tdH)
    assert torch.equal(dX, dX2) and torch.equal(dG, dG2)
