"""fp8_rope against the FP64 oracle.

Bound, derived before the first run: the angle in half turns is rounded to FP32
once it lies in [-1, 1] (2^-25; 2^-23 radians at most), sine and cosine add 2 ulp (2^-23), the
amplitude, the products and the sum a rounding each (4 x 2^-24 of the terms), the type half a step:
  |got - ref| <= eps / 2 |ref| + amplitude (|x1| + |x2|) 2^-21
(finfo(t).eps / 2: bf16 2^-8, f32 2^-24)
"""

import numpy as np
import pytest

from oracle import layer
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.double().cpu().numpy()


def _check(got, x, pos, freq, amplitude, interleaved, backward):
    import torch
    X = _f64(x)
    ref = layer.rope(X, pos, freq, amplitude, interleaved, backward)
    size = np.abs(X)
    mate = size.copy()
    r = 2 * len(freq)
    if interleaved:
        mate[..., 0:r:2], mate[..., 1:r:2] = size[..., 1:r:2], size[..., 0:r:2]
    else:
        mate[..., :r // 2], mate[..., r // 2:r] = size[..., r // 2:r], size[..., :r // 2]
    half = torch.finfo(got.dtype).eps / 2
    bound = half * np.abs(ref) + amplitude * (size + mate) * 2.0 ** -21
    g = _f64(got)
    assert np.all(np.abs(g - ref) <= bound), float(np.max(np.abs(g - ref) - bound))
    assert np.array_equal(g[..., r:], X[..., r:])


def _freq(rot, base=10000.0):
    return np.array([base ** (-2 * i / rot) for i in range(rot // 2)], np.float32)


@pytest.mark.parametrize("T,hq,hk,dim,rot,kind", [
    (1, 1, 1, 16, 16, "bf16"), (1, 64, 8, 128, 128, "bf16"), (3, 5, 1, 96, 48, "f32"), (7, 2, 2, 64, 32, "bf16"),
    (130, 8, 2, 256, 256, "f32"), (1001, 3, 0, 80, 80, "bf16"), (2, 4, 3, 512, 512, "f32"), (700, 12, 4, 128, 64, "bf16")])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("backward", [False, True])
def test_positions(T, hq, hk, dim, rot, kind, interleaved, backward):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    t = torch.bfloat16 if kind == "bf16" else torch.float32
    g = np.random.default_rng(T + dim)
    q, k = (dev(g.standard_normal((T, h, dim)).astype(np.float32)).to(t) for h in (hq, hk))
    pos = g.integers(0, 1 << 20, T).astype(np.int32)
    pos[0] = 0
    if T > 2:
        pos[1], pos[2] = 2 ** 31 - 1, -2 ** 31
    freq = _freq(rot)
    qo, ko = b.fp8_rope(q, k if hk else None, dev(freq), positions=dev(pos), interleaved=interleaved, amplitude=1.25,
                        backward=backward)
    _check(qo, q, pos, freq, 1.25, interleaved, backward)
    if hk:
        _check(ko, k, pos, freq, 1.25, interleaved, backward)
    else:
        assert ko is None
    assert b.fp8gemm_get_device_status() == b.OK


@pytest.mark.parametrize("new,old", [([1] * 5, [0, 7, 131071, 3, 64]), ([3, 0, 1, 300, 0, 17], [0, 5, 0, 1000, 2, 99]),
                                     ([2] * 100, list(range(100)))])
def test_parts_of_a_fused_row_at_the_end_of_sequences(new, old):
    """Ragged sequences, queries and keys as parts of wider rows, out of place and in place; with rows behind the
    last sequence, which stay."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    hq, hk, dim, spare = 4, 2, 64, 3
    T = sum(new)
    g = np.random.default_rng(T)
    fused = dev(g.standard_normal((T + spare, (hq + 2 * hk) * dim)).astype(np.float32)).to(torch.bfloat16)
    q, k, v = (x.unflatten(1, (-1, dim)) for x in fused.split([hq * dim, hk * dim, hk * dim], 1))
    lens = dev(np.array([a + n for a, n in zip(old, new)], np.int32))
    cu = dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
    pos = np.concatenate([a + np.arange(n) for a, n in zip(old, new)])
    freq = _freq(dim)
    qo, ko = (torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda") for x in (q, k))
    b.fp8_rope(q, k, dev(freq), seq_lens=lens, cu=cu, Qo=qo, Ko=ko)
    for got, x in ((qo, q), (ko, k)):
        _check(got[:T], x[:T], pos, freq, 1.0, False, False)
        assert bool((got[T:] == 7).all())
    if len(set(new)) == 1:
        same, _ = b.fp8_rope(q[:T], None, dev(freq), seq_lens=lens)
        assert torch.equal(same, qo[:T])
    before = fused.clone()
    b.fp8_rope(q, k, dev(freq), seq_lens=lens, cu=cu, Qo=q, Ko=k)
    assert torch.equal(q[:T], qo[:T]) and torch.equal(k[:T], ko[:T])
    assert torch.equal(fused[T:], before[T:]) and torch.equal(v, before[:, -hk * dim:].unflatten(1, (-1, dim)))
    assert b.fp8gemm_get_device_status() == b.OK


def test_partial_heads_in_place_and_part_of_the_head():
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = np.random.default_rng(3)
    x = dev(g.standard_normal((9, 3, 96)).astype(np.float32))
    pos, freq = np.arange(9, dtype=np.int32) * 1000, _freq(32)
    y = x.clone()
    b.fp8_rope(y, None, dev(freq), positions=dev(pos), interleaved=True, Qo=y)
    _check(y, x, pos, freq, 1.0, True, False)
    z = y.clone()
    b.fp8_rope(z, None, dev(freq), positions=dev(pos), interleaved=True, backward=True, Qo=z)
    assert float((z - x).abs().max()) <= 2.0 ** -20  # a rotation and back: two passes of the bound above


def test_gradient_against_differences():
    """sum(w y) along a direction: the inner product with the gradient (both linear: equal up to rounding)."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = np.random.default_rng(4)
    x, w, d = (dev(g.standard_normal((33, 4, 128)).astype(np.float32)) for _ in range(3))
    args = dict(positions=dev(g.integers(0, 99999, 33).astype(np.int32)), amplitude=1.1)
    f = dev(_freq(128))
    up, down = (b.fp8_rope(x + s * d, None, f, **args)[0] for s in (0.5, -0.5))
    diff = float((w.double() * (up.double() - down.double())).sum())
    grad = b.fp8_rope(w, None, f, backward=True, **args)[0]
    want = float((grad.double() * d.double()).sum())
    size = float((w.abs().double() * (x.abs() + d.abs()).double()).sum())
    assert abs(diff - want) <= 2.0 ** -19 * size


def test_bad_offsets_and_lengths_set_the_status():
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    q = torch.ones((6, 1, 32), device="cuda")
    f = dev(_freq(32))
    i32 = lambda *v: dev(np.array(v, np.int32))  # noqa: E731
    for lens, cu, touched in ((i32(9, 1), i32(0, 2, 6), 2), (i32(9, 9), i32(0, 2, 9), 2), (i32(9, 9), i32(0, -4, 3), 0)):
        out = torch.full_like(q, 5.0)
        b.fp8_rope(q, None, f, seq_lens=lens, cu=cu, Qo=out)
        assert b.fp8gemm_get_device_status() == b.ERR_DEVICE_STATUS
        assert bool((out[touched:] == 5).all()) and bool((out[:touched] != 5).all())
    b.fp8_rope(q[:0], None, f, seq_lens=i32())
    b.fp8_rope(q, None, f, seq_lens=i32(1, 1), cu=i32(0, 0, 0))  # no sequence has a token
    assert b.fp8gemm_get_device_status() == b.OK


def test_lengths_at_the_types_end():
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    q = torch.ones((6, 1, 32), device="cuda")
    f = dev(_freq(32))
    lens = dev(np.array([-2 ** 31, 2 ** 31 - 1], np.int32))
    cu = dev(np.array([0, 3, 6], np.int32))
    out = torch.full_like(q, 5.0)
    b.fp8_rope(q, None, f, seq_lens=lens, cu=cu, Qo=out)  # the first has fewer tokens than new ones
    assert b.fp8gemm_get_device_status() == b.ERR_DEVICE_STATUS
    assert bool((out[:3] == 5).all())
    same = b.fp8_rope(q[3:], None, f, positions=dev(np.array([2 ** 31 - 4, 2 ** 31 - 3, 2 ** 31 - 2], np.int32)))[0]
    assert torch.equal(out[3:], same)


@pytest.mark.parametrize("lens,cu", [
    ((9, 9, 9), (0, 4, 2, 6)), ((9, 9, 9), (0, 6, 3, 3)), ((9, 9), (-3, 0, 6)), ((9, 9), (0, 6, 9)), ((9, -1, 9), (0, 3, 3, 6)),
    ((9,) * 400 + (-7,), (0,) * 400 + (6, 6)), ((9,) * 300, (0,) * 150 + (-1,) * 150 + (6,))])
def test_every_sequence_is_looked_at(lens, cu):
    """Offsets that fall or leave the tokens, and lengths below 0, of sequences that no token finds."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    q = torch.ones((6, 1, 32), device="cuda")
    b.fp8_rope(q, None, dev(_freq(32)), seq_lens=dev(np.array(lens, np.int32)), cu=dev(np.array(cu, np.int32)))
    assert b.fp8gemm_get_device_status() == b.ERR_DEVICE_STATUS
    assert b.fp8gemm_get_device_status() == b.OK
