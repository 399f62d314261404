"""fp8_moe_few at sizes whose work is cut as large calls' is: runs of many K blocks that
begin and end anywhere in a tile, span several tiles and wrap each warp's ring, with 1,
2 and 4 fragments of tokens.

Against the formula in 64 bits.  Bounds, derived before the first run: a product's
FP32 sum (8 instructions a K block, at most 121 blocks or 160 partials) errs by less than
2^-17 of the sum of its terms' magnitudes; that moves h by d = |up| err(gate) 1.1 + |silu|
err(up) + 2^-20 |h|, and h's code to one between those of h - d' and h + d', d' = d + |h|
(d / |h| of the block's largest).  The output's bound is what those codes can differ by
through |W2|, 2^-17 of its own sum of magnitudes, and half a BF16 step twice over.
"""

import pytest

pytestmark = pytest.mark.gpu


def _operands(T, H, I, E, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def codes(*shape):  # random bytes, no NaN
        return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8, device="cuda") & 0xF7

    def scales(mean, *shape):
        return mean * (0.5 + torch.rand(shape, generator=g, device="cuda"))

    b = lambda n: -(-n // 128)  # noqa: E731
    return [codes(T, H), scales(1e-2, T, b(H)), torch.randn((T, E), generator=g, device="cuda"),
            codes(E, 2 * I, H), scales(1e-3 / H ** 0.5, E, b(2 * I), b(H)),
            codes(E, H, I), scales(1e-2, E, b(H), b(I))]


def _values(codes, scale):
    import torch
    v = codes.view(torch.float8_e4m3fn).double()
    s = scale.double()
    if v.shape[0] != s.shape[0]:
        s = s.repeat_interleave(128, 0)[:v.shape[0]]
    return v * s.repeat_interleave(128, 1)[:, :v.shape[1]]


def _code(x):
    import torch
    return x.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()


def _reference(ops, k):
    import torch
    A, sA, logits, W1, s1, W2, s2 = ops
    T, H = A.shape
    E, _, I = W2.shape
    x = _values(A, sA)
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.softmax(torch.gather(logits, 1, ids).double(), 1)
    out, slack = (torch.zeros((T, H), dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        w1, w2 = _values(W1[e], s1[e]), _values(W2[e], s2[e])
        u, err = x[t] @ w1.t(), 2.0 ** -17 * (x[t].abs() @ w1.abs().t())
        silu = u[:, :I] * torch.sigmoid(u[:, :I])
        h = silu * u[:, I:]
        d = 1.1 * err[:, :I] * u[:, I:].abs() + silu.abs() * err[:, I:] + 2.0 ** -20 * h.abs()
        q, dq = torch.zeros_like(h), torch.zeros_like(h)
        for c in range(0, I, 128):
            b, db = h[:, c:c + 128], d[:, c:c + 128]
            top, at = b.abs().max(1, keepdim=True)
            s = top / 448
            db = db + b.abs() * torch.gather(db, 1, at) / top
            q[:, c:c + 128] = _code(b / s) * s
            dq[:, c:c + 128] = (_code((b + db) / s) - _code((b - db) / s)).abs() * s + 2.0 ** -20 * b.abs()
        wt = w[t, j][:, None]
        out.index_add_(0, t, wt * (q @ w2.t()))
        slack.index_add_(0, t, wt * (dq @ w2.abs().t() + 2.0 ** -17 * (q.abs() @ w2.abs().t())))
    return out, slack + 2.0 ** -8 * out.abs(), ids


def _cut(T, H, I, E, k, ids):
    """(per, parts) of the up and of the down kernel, as they share their units out."""
    import torch
    b = lambda n: -(-n // 128)  # noqa: E731
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    nt = 1 if T <= 8 else 2 if T * k <= 32 * E else 4
    counts = torch.bincount(ids.flatten(), minlength=E).tolist()
    passes = sum(-(-n // (8 * nt)) for n in counts)
    cut = []
    for tiles, n in ((passes * b(I), b(H)), (b(H), passes * b(I))):
        per = max(2, -(-tiles * n // ((2 if nt == 4 else 3) * sms)))
        parts = n // per
        cut.append((per, 0 if parts > 0 and -(-n // parts) > per + 1 else parts))
    return cut


@pytest.mark.parametrize("T,H,I,E,k,uneven", [
    (1, 4112, 1920, 8, 8, 0), (24, 4112, 1920, 8, 2, 0), (64, 4112, 528, 8, 6, 0),
    (1, 15376, 528, 8, 8, 1), (24, 15376, 528, 8, 2, 1), (64, 10256, 528, 8, 6, 1),
    (8, 7168, 2048, 4, 4, None), (33, 2064, 3088, 16, 3, None)])
def test_moe_work_cut_as_large_calls_are(T, H, I, E, k, uneven):
    """uneven: which kernel's runs are not equal parts of a tile."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    ops = _operands(T, H, I, E, seed=T + H)
    out, bound, rids = _reference(ops, k)
    cut = _cut(T, H, I, E, k, rids)
    assert min(per for per, _ in cut) > 3  # more units in a run than a ring has stages
    if uneven is not None:
        assert cut[uneven][1] == 0
    D = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    D, ids, _ = b.fp8_moe_few(*ops, k, D=D)
    assert torch.equal(ids.long(), rids)
    bad = ~((D.double() - out).abs() <= bound)
    assert not bool(bad.any()), (int(bad.sum()), bad.numel(), D[bad][:4], out[bad][:4], bound[bad][:4])
    assert float(bound.median()) < 0.05 * float(out.square().mean().sqrt())  # the bound tells something
    assert torch.equal(b.fp8_moe_few(*ops, k)[0], D)
    assert b.fp8gemm_get_device_status() == b.OK
