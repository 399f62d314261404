"""fp8_moe_few against the FP64 oracle: routing equal, weights to FP32's
rounding (an exponential, a sum of at most 512 and a division: 2e-6 relative),
outputs within the GEMMs' acceptance (tests/gpu_helpers.py), and bit for bit
against itself."""

import numpy as np
import pytest

from oracle import layer
from tests.gpu_helpers import assert_close, dev, host, oquant, quant_weights

pytestmark = pytest.mark.gpu


def _operands(T, H, I, E, seed):
    g = np.random.default_rng(seed)
    A, sA = oquant.quant_1x128_fast(g.standard_normal((T, H)).astype(np.float32))
    W = [[quant_weights((0.05 * g.standard_normal(s)).astype(np.float32)) for s in ((2 * I, H), (H, I))]
         for _ in range(E)]
    W1, s1 = (np.stack([w[0][i] for w in W]) for i in (0, 1))
    W2, s2 = (np.stack([w[1][i] for w in W]) for i in (0, 1))
    return [A, sA, (2 * g.standard_normal((T, E))).astype(np.float32), W1, s1, W2, s2]


def _check(ops, k, renormalise=True):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    t = [dev(x) for x in ops]
    D = torch.full((ops[0].shape[0], ops[0].shape[1]), float("nan"), dtype=torch.bfloat16, device="cuda")
    D, ids, w = b.fp8_moe_few(*t, k, renormalise=renormalise, D=D)
    out, rids, rw = layer.moe(*ops, k, renormalise)
    assert np.array_equal(host(ids), rids)
    assert np.all(np.abs(host(w) - rw) <= 2e-6 * rw + 1e-30)
    assert_close(host(D), out, "moe")
    D2, _, _ = b.fp8_moe_few(*t, k, renormalise=renormalise)
    assert torch.equal(D, D2)
    assert b.fp8gemm_get_device_status() == b.OK


@pytest.mark.parametrize("T,H,I,E,k,renormalise", [
    (1, 16, 16, 1, 1, True), (1, 128, 128, 4, 2, True), (1, 1040, 400, 9, 4, False), (2, 256, 144, 3, 3, True),
    (7, 400, 208, 40, 8, True), (8, 512, 256, 2, 1, True), (9, 272, 528, 5, 2, False), (16, 256, 384, 6, 16 // 4, True),
    (17, 144, 128, 1, 1, True), (33, 384, 256, 8, 2, True), (64, 256, 272, 4, 4, True), (64, 512, 128, 16, 2, True),
    (3, 128, 64, 300, 16, False)])
def test_moe(T, H, I, E, k, renormalise):
    _check(_operands(T, H, I, E, seed=T + H + I + E), k, renormalise)


def test_all_tokens_on_one_expert():
    ops = _operands(64, 256, 256, 5, seed=1)
    ops[2][:, 3] = 50
    _check(ops, 1)


def test_ties_bans_and_nan():
    ops = _operands(6, 256, 128, 8, seed=2)
    lg = ops[2]
    lg[0] = 0                       # all tied
    lg[1, :6] = -np.inf             # two left
    lg[2, [1, 5]] = np.nan          # never chosen
    lg[3] = 1e30
    lg[4] = np.float32(-3e38)       # the type's lowest region, all tied
    lg[5, 7] = 90
    _check(ops, 2)


def test_banned_experts_get_weight_zero():
    from fp8_fine_grained_e4m3_gb300 import binding as b
    ops = _operands(2, 128, 128, 4, seed=3)
    ops[2][0, 1:] = -np.inf
    ops[2][1] = -np.inf
    D, ids, w = b.fp8_moe_few(*[dev(x) for x in ops], 3)
    assert host(ids).tolist() == [[0, 1, 2], [0, 1, 2]]
    assert host(w).tolist() == [[1, 0, 0], [0, 0, 0]]
    assert np.isfinite(host(D)).all() and not host(D)[1].any()


def test_matches_the_grouped_calls():
    """The same layer out of the grouped GEMM, SwiGLU in torch and the quantiser."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    T, H, I, E = 24, 512, 256, 3
    ops = _operands(T, H, I, E, seed=4)
    A, sA, lg, W1, s1, W2, s2 = [dev(x) for x in ops]
    D, ids, w = b.fp8_moe_few(A, sA, lg, W1, s1, W2, s2, 1)
    mi = torch.full((E, 128), -1, dtype=torch.int32, device="cuda")
    Ap = torch.zeros((E, 128, H), dtype=torch.uint8, device="cuda")
    sp = torch.zeros((E, 128, H // 128), device="cuda")
    for e in range(E):
        t = torch.nonzero(ids[:, 0] == e).flatten()
        mi[e, :len(t)] = e
        Ap[e, :len(t)], sp[e, :len(t)] = A[t], sA[t]
    u = b.fp8gemm_grouped_contiguous(Ap.view(-1, H), sp.view(-1, H // 128), W1, s1, mi.view(-1)).float()
    h = torch.where(mi.view(-1, 1) >= 0, torch.nn.functional.silu(u[:, :I]) * u[:, I:], 0)
    h8, sh = b.fp8_quant_1x128(h.contiguous())
    y = b.fp8gemm_grouped_contiguous(h8, sh, W2, s2, mi.view(-1)).view(E, 128, H)
    ref = torch.zeros((T, H), device="cuda")
    for e in range(E):
        t = torch.nonzero(ids[:, 0] == e).flatten()
        ref[t] = y[e, :len(t)].float()
    # the chain rounds u and y to BF16 on the way and re-rounds h to FP8: a few percent of a typical element
    err = (D.float() - ref).norm() / ref.norm()
    assert float(err) < 0.05


def test_calls_back_to_back_on_two_streams():
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    a, c = (([dev(x) for x in _operands(T, 512, 256, 6, seed=T)]) for T in (3, 40))
    want = [b.fp8_moe_few(*x, 2)[0] for x in (a, c)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(6):
        got.append((i % 2, b.fp8_moe_few(*(a, c)[i % 2], 2, stream=streams[i // 2 % 2])[0]))
    torch.cuda.synchronize()
    for i, D in got:
        assert torch.equal(D, want[i])
    for s in streams:
        b.fp8gemm_release_workspaces(s)


@pytest.mark.parametrize("T,k", [(1, 8), (40, 1)])
def test_a_wait_that_runs_out_is_reported(T, k):
    """Weights of more than the L2, few tokens for each of them and a 1 ns limit:
    waits for their copies are genuine, the layer gives up and says so; the
    next call is right."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    H, I, E = 7168, 2048, 8
    W1 = torch.randint(0, 100, (E, 2 * I, H), dtype=torch.uint8, device="cuda")
    W2 = torch.randint(0, 100, (E, H, I), dtype=torch.uint8, device="cuda")
    s1, s2 = (torch.full(s, 1e-3, device="cuda") for s in ((E, 2 * I // 128, H // 128), (E, H // 128, I // 128)))
    A = torch.randint(0, 256, (T, H), dtype=torch.uint8, device="cuda") & 0xF7  # no NaN
    sA = torch.full((T, H // 128), 1e-2, device="cuda")
    args = (A, sA, torch.randn((T, E), device="cuda"), W1, s1, W2, s2, k)
    want = b.fp8_moe_few(*args)[0]
    torch.cuda.synchronize()
    b.set_wait_limit_ns(1)
    try:
        b.fp8_moe_few(*args)
        assert b.fp8gemm_get_device_status() == b.ERR_TIMEOUT
    finally:
        b.set_wait_limit_ns(0)
    assert torch.equal(b.fp8_moe_few(*args)[0], want)
    assert b.fp8gemm_get_device_status() == b.OK


@pytest.mark.parametrize("scale", [1e-32, 1e30])
def test_extreme_hidden_scales(scale):
    """Hidden activations whose block scale is far from 1: the corrected quotient
    works on values brought into its range."""
    ops = _operands(3, 256, 128, 3, seed=9)
    ops[4] = (ops[4] * np.float32(np.sqrt(scale))).astype(np.float32)
    ops[6] = (ops[6] / np.float32(scale)).astype(np.float32)
    _check(ops, 2)


def test_more_calls_of_other_sizes_share_a_workspace():
    """Small and large calls in turn on one stream: the counters a call leaves
    are zeros wherever the next one's buffers lie."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    sets = [[dev(x) for x in _operands(T, H, I, E, seed=T)] for T, H, I, E in
            ((1, 128, 128, 2), (64, 512, 256, 8), (7, 1040, 400, 9), (20, 256, 128, 3))]
    want = []
    for s in sets:
        b.fp8gemm_release_workspaces()
        want.append(b.fp8_moe_few(*s, 2)[0].clone())
    for _ in range(3):
        for s, w in zip(sets, want):
            assert torch.equal(b.fp8_moe_few(*s, 2)[0], w)


def test_a_hidden_scale_that_underflows():
    """|h| of 1e-44 to 3e-43: max |h| / 448 is 0 in FP32.  The codes are zeros and
    the token's output is 0, for a token beside others that are ordinary too."""
    from fp8_fine_grained_e4m3_gb300 import binding as b
    ops = _operands(3, 256, 128, 3, seed=10)
    ops[4] = (ops[4] * np.float32(2e-22)).astype(np.float32)
    D, _, _ = b.fp8_moe_few(*[dev(x) for x in ops], 2)
    assert (host(D) == 0).all()
    ops = _operands(3, 256, 128, 3, seed=11)
    ops[1][1] *= np.float32(2e-22)
    _check(ops, 2)
    D, _, _ = b.fp8_moe_few(*[dev(x) for x in ops], 2)
    assert (host(D)[1] == 0).all()
