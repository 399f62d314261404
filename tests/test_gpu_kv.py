"""fp8_kv_append bit for bit, and fp8_kv_attention within its rounding,
against the FP64 oracle.

Attention's bound, derived before the first run: p is rounded to FP16 (2^-11
relative, or 2^-25 of the largest p absolute), the scores and sums are FP32
(together under 2^-12 relative here), the output BF16 (2^-9 relative):
  |got - ref| <= 2^-8 |ref| + 2^-10 sum p |v| + n 2^-24 max |v|
"""

import numpy as np
import pytest

from oracle import layer
from tests.gpu_helpers import dev, host

pytestmark = pytest.mark.gpu

_CODES = {"e4m3": layer.e4m3, "e5m2": layer.e5m2}


class Cache:
    """A paged cache with codes everywhere, and NaN codes behind each sequence."""

    def __init__(self, lens, heads, dim, block, fmt, seed, spread=2, spare=2):
        g = np.random.default_rng(seed)
        per = [-(-n // block) for n in lens]
        self.n, self.width = max(1, sum(per)) + spare, max(1, max(per))
        order = g.permutation(self.n)
        self.table = np.zeros((len(lens), self.width), np.int32)
        at = 0
        for b, p in enumerate(per):
            self.table[b, :p] = order[at:at + p]
            at += p
        enc = _CODES[fmt].encode_rne_sat
        limit = 448.0 if fmt == "e4m3" else 57344.0
        shape = (self.n, heads, block, dim)
        self.k, self.v = (enc((limit / 5 * g.standard_normal(shape)).astype(np.float32)) for _ in range(2))
        self.ks, self.vs = (np.exp2(g.integers(-spread, spread + 1, (self.n, heads)) - np.round(np.log2(limit / 5)))
                            .astype(np.float32) for _ in range(2))
        self.lens, self.fmt = np.asarray(lens, np.int32), fmt

    def stale(self):
        used = {int(x) for b, n in enumerate(self.lens) for x in self.table[b, :-(-n // self.k.shape[2])]}
        for x in (self.k, self.v):
            for b, n in enumerate(self.lens):
                if n % x.shape[2]:
                    x[self.table[b, n // x.shape[2]], :, n % x.shape[2]:] = 0x7F
            for blk in set(range(self.n)) - used:
                x[blk] = 0x7F
        return self

    def on_gpu(self):
        return [dev(x) for x in (self.k, self.ks, self.v, self.vs, self.table, self.lens)]


def _offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_append(block, dim, fmt):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    new = [1, 0, 3, 150, 17, 1, 64]
    old = [0, 5, 15, 7, 128, 200, 64]
    heads = 3
    c = Cache([a + n for a, n in zip(old, new)], heads, dim, block, fmt, seed=block + dim)
    g = np.random.default_rng(1)
    T = sum(new)
    cu = _offsets(new)
    wide = (np.exp2(g.integers(-6, 7, (T, 1))) * g.standard_normal((T, 3 * heads * dim))).astype(np.float32)
    wide[5:60] = 0  # whole blocks of zeros
    qkv = dev(wide).to(torch.bfloat16)
    w = heads * dim
    K, V = (qkv[:, i * w:(i + 1) * w].unflatten(1, (heads, dim)) for i in (1, 2))
    k, ks, v, vs, table, lens = c.on_gpu()
    b.fp8_kv_append(K, V, k, ks, v, vs, table, lens, cu_new=dev(cu), max_new=max(new), fmt=fmt)
    layer.kv_append(K.float().cpu().numpy(), c.k, c.ks, c.table, c.lens, cu, fmt)
    layer.kv_append(V.float().cpu().numpy(), c.v, c.vs, c.table, c.lens, cu, fmt)
    for got, ref in ((k, c.k), (ks, c.ks), (v, c.v), (vs, c.vs)):
        assert np.array_equal(host(got), ref)
    assert b.fp8gemm_get_device_status() == b.OK


def test_append_token_by_token_grows_scales():
    """A sequence written one token at a time, ever larger: every step requantises."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    heads, dim, block = 2, 128, 16
    c = Cache([40], heads, dim, block, "e4m3", seed=2)
    k, ks, v, vs, table, _ = c.on_gpu()
    g = np.random.default_rng(3)
    for n in range(1, 41):
        x = dev((1.7 ** (n % 20) * g.standard_normal((1, heads, dim))).astype(np.float32)).to(torch.bfloat16)
        b.fp8_kv_append(x, -x, k, ks, v, vs, table, dev(np.array([n], np.int32)))
        layer.kv_append(x.float().cpu().numpy(), c.k, c.ks, c.table, [n], [0, 1])
        layer.kv_append(-x.float().cpu().numpy(), c.v, c.vs, c.table, [n], [0, 1])
    for got, ref in ((k, c.k), (ks, c.ks), (v, c.v), (vs, c.vs)):
        assert np.array_equal(host(got), ref)


def _attend(c, Q, cu, scale, fmt, **kw):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    tQ = dev(Q).to(torch.bfloat16)
    k, ks, v, vs, table, lens = c.on_gpu()
    O = torch.full(tQ.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    b.fp8_kv_attention(tQ, k, ks, v, vs, table, lens, cu_q=None if cu is None else dev(cu), scale=scale, fmt=fmt,
                       O=O, **kw)
    return host(O), tQ.double().cpu().numpy()


def _check(got, c, Q, cu, scale, fmt):
    O, A = layer.kv_attention(Q, c.k, c.ks, c.v, c.vs, c.table, c.lens, cu, scale, fmt)
    vmax = np.nanmax(np.abs(_CODES[fmt].decode(c.v)) * c.vs[:, :, None, None].astype(np.float64))
    bound = 2.0 ** -8 * np.abs(O) + 2.0 ** -10 * A + max(c.lens.max(), 1) * 2.0 ** -24 * vmax
    bad = ~(np.abs(got - O) <= bound)
    assert not bad.any(), (int(bad.sum()), bad.size, got[bad][:4], O[bad][:4])


@pytest.mark.parametrize("lens,heads,group,dim,block,fmt,q", [
    ([1], 1, 1, 64, 16, "e4m3", 1), ([37], 2, 1, 64, 16, "e4m3", 1), ([0, 5, 300, 16], 2, 3, 128, 32, "e4m3", 1),
    ([1000, 17, 64], 2, 8, 128, 64, "e4m3", 1), ([511, 2], 1, 16, 128, 128, "e5m2", 1),
    ([200, 3, 0, 65], 3, 5, 64, 64, "e5m2", 4), ([130, 2, 77], 2, 4, 128, 16, "e4m3", 7),
    ([4099], 2, 8, 128, 64, "e4m3", 2), ([600, 601], 1, 8, 128, 32, "e4m3", 20), ([33] * 70, 2, 2, 64, 16, "e4m3", 1)])
def test_attention(lens, heads, group, dim, block, fmt, q):
    c = Cache(lens, heads, dim, block, fmt, seed=sum(lens)).stale()
    g = np.random.default_rng(7)
    Q = (2 * g.standard_normal((len(lens) * q, heads * group, dim))).astype(np.float32)
    cu = _offsets([q] * len(lens))
    got, Qr = _attend(c, Q, None, dim ** -0.5, fmt)
    _check(got, c, Qr, cu, dim ** -0.5, fmt)
    got2, _ = _attend(c, Q, cu, dim ** -0.5, fmt, max_q=q)
    assert np.array_equal(got, got2)


def test_attention_of_ragged_queries_from_a_fused_row():
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    counts, heads, group, dim = [3, 0, 1, 9, 2], 2, 4, 128
    c = Cache([70, 10, 1, 9, 1], heads, dim, 32, "e4m3", seed=5).stale()  # the last: one token, two queries
    cu = _offsets(counts)
    g = np.random.default_rng(6)
    w = heads * group * dim
    qkv = dev(g.standard_normal((sum(counts), w + 2 * heads * dim)).astype(np.float32)).to(torch.bfloat16)
    tQ = qkv[:, :w].unflatten(1, (heads * group, dim))
    k, ks, v, vs, table, lens = c.on_gpu()
    O = b.fp8_kv_attention(tQ, k, ks, v, vs, table, lens, cu_q=dev(cu), max_q=9, scale=0.3)
    _check(host(O), c, tQ.double().cpu().numpy(), cu, 0.3, "e4m3")
    assert not O[cu[4]].any()  # sees nothing


@pytest.mark.parametrize("kind", ["peaked", "flat", "rising", "falling", "tiny_q", "huge_q", "wide_scales"])
def test_attention_statistics(kind):
    """Scores that one token dominates, that are all equal, that rise or fall
    along the cache, queries near the ends of BF16's range, and scales of
    neighbouring blocks that differ by 2^40."""
    heads, dim, n = 1, 128, 700
    c = Cache([n], heads, dim, 16, "e4m3", seed=9, spread=20 if kind == "wide_scales" else 1)
    g = np.random.default_rng(10)
    Q = g.standard_normal((1, 8, dim)).astype(np.float32)
    scale = dim ** -0.5
    enc = layer.e4m3.encode_rne_sat
    if kind == "peaked":
        c.k[c.table[0, 20], 0, 3] = enc((50 * np.sign(Q[0, 0])).astype(np.float32))
        Q[:] = Q[:, :1]
        scale = 1.0
    elif kind == "flat":
        Q[:] = 0
    elif kind in ("rising", "falling"):
        ramp = np.linspace(-1, 1, c.width * 16).astype(np.float32) * (1 if kind == "rising" else -1)
        for j in range(c.width):
            c.k[c.table[0, j], 0] = enc(np.repeat(400 * ramp[16 * j:16 * j + 16, None], dim, 1))
        c.ks[:] = 2.0 ** -9
        Q[:] = 8
    elif kind == "tiny_q":
        Q *= 1e-30
        scale = 1e29
    elif kind == "huge_q":
        Q *= 1e30
        scale = 1e-31
    elif kind == "wide_scales":
        c.ks[:] = 2.0 ** -6
    got, Qr = _attend(c, Q, None, scale, "e4m3")
    _check(got, c, Qr, [0, 1], scale, "e4m3")


def test_long_cache_past_32_bit_offsets():
    """A cache whose byte offsets pass 2^32, the sequence in its last blocks."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    heads, dim, block = 8, 128, 128
    n = 2 ** 32 // (heads * dim * block) + 40
    c = Cache([1500], heads, dim, block, "e4m3", seed=12, spare=0)
    k, v = (torch.zeros((n, heads, block, dim), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((n, heads), device="cuda") for _ in range(2))
    far = n - c.n
    k[far:], v[far:], ks[far:], vs[far:] = dev(c.k), dev(c.v), dev(c.ks), dev(c.vs)
    g = np.random.default_rng(13)
    tQ, tK, tV = (dev(g.standard_normal((1, h, dim)).astype(np.float32)).to(torch.bfloat16) for h in (16, 8, 8))
    table, lens = dev(c.table + far), dev(c.lens)
    b.fp8_kv_append(tK, tV, k, ks, v, vs, table, lens)
    O = b.fp8_kv_attention(tQ, k, ks, v, vs, table, lens)
    layer.kv_append(tK.float().cpu().numpy(), c.k, c.ks, c.table, c.lens, [0, 1])
    layer.kv_append(tV.float().cpu().numpy(), c.v, c.vs, c.table, c.lens, [0, 1])
    assert np.array_equal(host(k[far:]), c.k) and np.array_equal(host(v[far:]), c.v)
    _check(host(O), c, tQ.double().cpu().numpy(), [0, 1], dim ** -0.5, "e4m3")


def test_bad_indices_set_the_status_and_touch_nothing():
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    c = Cache([40, 50], 1, 64, 16, "e4m3", seed=20)
    g = np.random.default_rng(21)
    x = dev(g.standard_normal((2, 1, 64)).astype(np.float32)).to(torch.bfloat16)
    k, ks, v, vs, table, lens = c.on_gpu()
    before = k.clone()

    def expect(call):
        call()
        assert b.fp8gemm_get_device_status() == b.ERR_DEVICE_STATUS

    bad = table.clone()
    bad[:, -2:] = torch.tensor([c.n, -1], device="cuda", dtype=torch.int32)
    expect(lambda: b.fp8_kv_append(x, x, k, ks, v, vs, bad, lens))
    expect(lambda: b.fp8_kv_append(x, x, k, ks, v, vs, table, torch.full_like(lens, 10 ** 6)))
    expect(lambda: b.fp8_kv_append(x, x, k, ks, v, vs, table, torch.zeros_like(lens)))
    cu = dev(np.array([0, 3, 2], np.int32))
    expect(lambda: b.fp8_kv_append(x, x, k, ks, v, vs, table, lens, cu_new=cu))
    assert torch.equal(k, before)
    expect(lambda: b.fp8_kv_attention(x, k, ks, v, vs, table, lens, cu_q=cu))
    O = None

    def run():
        nonlocal O
        O = b.fp8_kv_attention(x, k, ks, v, vs, table, torch.tensor([-3, 10 ** 6], device="cuda", dtype=torch.int32))
    expect(run)
    assert not O.any()
    expect(lambda: b.fp8_kv_attention(x, k, ks, v, vs, torch.full_like(table, c.n), lens))
    expect(lambda: b.fp8_kv_attention(x, k, ks, v, vs, torch.full_like(table, -1), lens))
    assert b.fp8gemm_get_device_status() == b.OK


def test_graph_replay_with_new_lengths():
    """A captured append and attention replayed with other lengths, tables and
    tokens equals the calls made directly."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    heads, group, dim, block, B = 2, 4, 128, 32, 3
    c = Cache([500, 400, 300], heads, dim, block, "e4m3", seed=30)
    g = np.random.default_rng(31)

    def inputs():
        return [dev(g.standard_normal((B, h, dim)).astype(np.float32)).to(torch.bfloat16)
                for h in (heads * group, heads, heads)]

    q, kn, vn = inputs()
    k, ks, v, vs, table, lens = c.on_gpu()
    mine = [x.clone() for x in (k, ks, v, vs)]
    O = torch.empty_like(q)

    def step(cache, o):
        b.fp8_kv_append(kn, vn, *cache, table, lens)
        b.fp8_kv_attention(q, *cache, table, lens, O=o)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step([k, ks, v, vs], O)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step([k, ks, v, vs], O)
    for a, x in zip((k, ks, v, vs), mine):
        a.copy_(x)
    for new in ([100, 399, 1], [101, 400, 2], [500, 33, 64]):
        lens.copy_(dev(np.array(new, np.int32)))
        for a, x in zip((q, kn, vn), inputs()):
            a.copy_(x)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        want = torch.empty_like(O)
        step(mine, want)
        assert torch.equal(O, want)
        for a, x in zip((k, ks, v, vs), mine):
            assert torch.equal(a, x)


def test_append_of_ragged_prompts_finds_its_tiles():
    """Many more places than tiles (one long prompt among short ones): the tiles
    are found by a running sum, over more than 32 sequences."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    new = [0, 1, 300] + [2, 0, 17] * 14
    old = [5] * len(new)
    c = Cache([a + n for a, n in zip(old, new)], 2, 64, 16, "e4m3", seed=40)
    g = np.random.default_rng(41)
    cu, T = _offsets(new), sum(new)
    K, V = (dev(g.standard_normal((T, 2, 64)).astype(np.float32)).to(torch.bfloat16) for _ in range(2))
    k, ks, v, vs, table, lens = c.on_gpu()
    b.fp8_kv_append(K, V, k, ks, v, vs, table, lens, cu_new=dev(cu), max_new=300)
    layer.kv_append(K.float().cpu().numpy(), c.k, c.ks, c.table, c.lens, cu)
    layer.kv_append(V.float().cpu().numpy(), c.v, c.vs, c.table, c.lens, cu)
    for got, ref in ((k, c.k), (ks, c.ks), (v, c.v), (vs, c.vs)):
        assert np.array_equal(host(got), ref)
    bad = lens.clone()
    bad[40] = -1
    b.fp8_kv_append(K, V, k, ks, v, vs, table, bad, cu_new=dev(cu), max_new=300)
    assert b.fp8gemm_get_device_status() == b.ERR_DEVICE_STATUS


def test_append_to_a_cache_with_other_scales():
    """A block filled by other means may hold any scale: not a power of two, and kept
    where it is large enough."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    c = Cache([40, 40], 1, 64, 64, "e4m3", seed=42)
    c.ks[:], c.vs[:] = 0.3, 1e-30
    g = np.random.default_rng(43)
    X = dev(g.standard_normal((2, 1, 64)).astype(np.float32)).to(torch.bfloat16)
    k, ks, v, vs, table, lens = c.on_gpu()
    b.fp8_kv_append(X, X, k, ks, v, vs, table, lens)
    for codes, s, got, gs in ((c.k, c.ks, k, ks), (c.v, c.vs, v, vs)):
        layer.kv_append(X.float().cpu().numpy(), codes, s, c.table, c.lens, [0, 1, 2])
        assert np.array_equal(host(got), codes) and np.array_equal(host(gs), s)


@pytest.mark.parametrize("B,heads,group,q,longest", [
    (1, 1, 8, 1, 9000), (1, 8, 4, 4, 5000), (3, 2, 1, 1, 3000), (40, 4, 2, 1, 700), (64, 3, 8, 2, 400),
    (19, 8, 1, 1, 900), (200, 1, 4, 1, 300)])
def test_attention_shared_among_ctas(B, heads, group, q, longest):
    """Few items in many parts and many items in runs, sequences of very
    different lengths among them: against the oracle on sampled rows, and bit
    for bit on a second call."""
    import torch
    g = np.random.default_rng(B)
    lens = [longest] + [int(x) for x in g.integers(0, longest, B - 1)]
    dim = 128
    c = Cache(lens, heads, dim, 32, "e4m3", seed=B + heads).stale()
    Q = g.standard_normal((B * q, heads * group, dim)).astype(np.float32)
    got, Qr = _attend(c, Q, None, dim ** -0.5, "e4m3")
    got2, _ = _attend(c, Q, None, dim ** -0.5, "e4m3")
    assert np.array_equal(got, got2)
    pick = sorted(set([0, B - 1] + [int(x) for x in g.integers(0, B, 4)]))
    table, clens = c.table, c.lens
    for b_ in pick:
        c.table, c.lens = table[b_:b_ + 1], clens[b_:b_ + 1]
        _check(got[b_ * q:(b_ + 1) * q], c, Qr[b_ * q:(b_ + 1) * q], [0, q], dim ** -0.5, "e4m3")


@pytest.mark.parametrize("B,length", [(1, 262144), (64, 4096)])
def test_a_wait_that_runs_out_is_reported(B, length):
    """A cache four times the L2 and a 1 ns limit: waits for its copies are
    genuine, the attention gives up and says so; the next call is right."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    heads, dim, block = 8, 128, 64
    n = B * length // block
    k, v = (torch.randint(0, 120, (n, heads, block, dim), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((n, heads), 2.0 ** -7, device="cuda") for _ in range(2))
    table = torch.randperm(n, device="cuda").to(torch.int32).view(B, -1)
    lens = torch.full((B,), length, dtype=torch.int32, device="cuda")
    q = torch.randn((B, heads * 2, dim), device="cuda").to(torch.bfloat16)
    want = b.fp8_kv_attention(q, k, ks, v, vs, table, lens)
    torch.cuda.synchronize()
    b.set_wait_limit_ns(1)
    try:
        b.fp8_kv_attention(q, k, ks, v, vs, table, lens)
        assert b.fp8gemm_get_device_status() == b.ERR_TIMEOUT
    finally:
        b.set_wait_limit_ns(0)
    assert torch.equal(b.fp8_kv_attention(q, k, ks, v, vs, table, lens), want)
    assert b.fp8gemm_get_device_status() == b.OK


@pytest.mark.parametrize("counts,group,heads,dim,block,fmt", [
    ([1], 17, 1, 128, 64, "e4m3"), ([4, 1, 2, 3], 8, 2, 128, 16, "e4m3"), ([11, 0, 1], 3, 5, 64, 32, "e5m2"),
    ([8] * 24, 5, 8, 128, 16, "e4m3"), ([5, 1, 3] * 20, 4, 8, 64, 128, "e4m3"), ([65, 2], 1, 2, 128, 32, "e5m2")])
def test_attention_of_more_rows_than_a_warp_takes(counts, group, heads, dim, block, fmt):
    """More than 16 rows for a cached head, up to many times that, next to
    sequences with few or none; few items and many."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    g = np.random.default_rng(len(counts) + group)
    lens = [n + int(x) for n, x in zip(counts, g.integers(0, 900, len(counts)))]
    lens[0] = 1237
    c = Cache(lens, heads, dim, block, fmt, seed=group).stale()
    cu = _offsets(counts)
    Q = (2 * g.standard_normal((sum(counts), heads * group, dim))).astype(np.float32)
    got, Qr = _attend(c, Q, cu, dim ** -0.5, fmt, max_q=max(counts))
    _check(got, c, Qr, cu, dim ** -0.5, fmt)
    assert np.array_equal(got, _attend(c, Q, cu, dim ** -0.5, fmt, max_q=max(counts))[0])
    assert b.fp8gemm_get_device_status() == b.OK


@pytest.mark.parametrize("dim,group,fmt", [(128, 1, "e4m3"), (64, 4, "e5m2"), (128, 16, "e4m3")])
@pytest.mark.parametrize("apart", [20, -20, 60])
def test_attention_keeps_the_smaller_of_two_scales(dim, group, fmt, apart):
    """Blocks of 16, two to a tile, whose value scales differ by 2^20 or 2^60, all the
    probability on every other one.  Bound relative to those: the others' p is below
    2^-100 by construction, so the terms of FP16's range above do not arise."""
    c = Cache([16 * 41], 1, dim, 16, fmt, seed=50, spread=0)
    enc, limit = _CODES[fmt].encode_rne_sat, 448.0 if fmt == "e4m3" else 57344.0
    lead = c.table[0, :c.width]
    c.k[lead[::2]], c.k[lead[1::2]] = enc(np.float32(limit)), enc(np.float32(-limit))  # scores of one sign each
    c.ks[:] = 1 / limit
    c.vs[lead[1::2]] *= np.float32(2.0 ** apart)
    Q = np.full((1, group, dim), 1.0, np.float32)
    got, Qr = _attend(c, Q, None, 100.0 / dim, fmt)  # scores +-100
    O, A = layer.kv_attention(Qr, c.k, c.ks, c.v, c.vs, c.table, c.lens, [0, 1], 100.0 / dim, fmt)
    assert np.all(np.abs(got - O) <= 2.0 ** -8 * np.abs(O) + 2.0 ** -10 * A)
    assert np.abs(O).max() > 0.01


@pytest.mark.parametrize("dim", [64, 128])
def test_attention_over_falling_scales(dim):
    """Value scales 1, 2^-59 and 2^-118 along a sequence, 384 tokens each in turn and
    long enough for a warp to meet all three one after the other: finite throughout."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    n, block = 150000, 32
    nb = -(-n // block)
    g = torch.Generator(device="cuda")
    g.manual_seed(51)
    k, v = (torch.randint(lo, 0x7F, (nb, 1, block, dim), generator=g, dtype=torch.uint8, device="cuda") for lo in (0, 0x60))
    ks = torch.full((nb, 1), 2.0 ** -7, device="cuda")
    vs = torch.exp2(-59.0 * (torch.arange(nb, device="cuda") // 12 % 3))[:, None]
    table = torch.arange(nb, dtype=torch.int32, device="cuda")[None]
    q = (0.01 * torch.randn((1, 2, dim), generator=g, device="cuda")).to(torch.bfloat16)
    got = b.fp8_kv_attention(q, k, ks, v, vs, table, torch.tensor([n], dtype=torch.int32, device="cuda")).double()
    deq = lambda c, s: (c.view(torch.float8_e4m3fn).double() * s.double()[..., None, None]).view(-1, dim)[:n]  # noqa: E731
    p = torch.softmax(q[0].double() @ deq(k, ks).t() * dim ** -0.5, 1)
    O = p @ deq(v, vs)  # values are positive: O is its own sum of magnitudes
    assert bool(((got[0] - O).abs() <= (2.0 ** -8 + 2.0 ** -10) * O + n * 2.0 ** -36 * 448).all())


@pytest.mark.parametrize("tail", [18.4, 14.0, 20.8])
@pytest.mark.parametrize("heads", [1, 40])
def test_attention_of_a_flat_tail_below_a_peak(tail, heads):
    """One token above 131072 others of equal scores and values of one sign, e^tail
    times as probable as each (2^26.5, 2^20, 2^30 times), its own value 0: the output is the
    tail alone.  p's rounding is 2^-12 relative, or, next to FP16's end, half of its
    least step, 2^-25, under the factor 2^11 that p is held with: 2^-36 of the peak a token."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    dim, n, block = 128, 131073, 128
    nb = -(-n // block)
    k = torch.zeros((nb, heads, block, dim), dtype=torch.uint8, device="cuda")
    v = torch.full_like(k, 0x70)  # 128
    k[77, :, 5], v[77, :, 5] = 0x38, 0  # 1
    ks, vs = (torch.full((nb, heads), x, device="cuda") for x in (1.0, 2.0 ** -7))
    table = torch.arange(nb, dtype=torch.int32, device="cuda")[None]
    scale = float(np.float32(tail / dim))
    got = host(b.fp8_kv_attention(torch.ones((1, heads, dim), device="cuda").to(torch.bfloat16), k, ks, v, vs, table,
                                  torch.tensor([n], dtype=torch.int32, device="cuda"), scale=scale))
    p = np.exp(-scale * dim)
    O, v = (n - 1) * p / (1 + (n - 1) * p), 1.0
    assert np.all(np.abs(got - O) <= 2.0 ** -8 * O + 2.0 ** -10 * O + n * 2.0 ** -36 * v)
    assert O > 4 * n * 2.0 ** -36 * v


@pytest.mark.parametrize("height", [2.0 ** 24, 1.7e8, 3e9])
def test_attention_of_scores_past_fp32_s_whole_numbers(height):
    """Scores whose spacing in FP32 is 1 to 256: the lift of p must not be lost in them.
    Equal ones give the mean of their values, whatever they round to."""
    dim = 64
    c = Cache([700], 3, dim, 32, "e4m3", seed=54, spread=0)
    c.k[:] = layer.e4m3.encode_rne_sat(np.float32(1))
    c.ks[:] = 1
    Q = np.full((1, 24, dim), 1.0, np.float32)
    got, Qr = _attend(c, Q, None, height / dim, "e4m3")
    _check(got, c, Qr, [0, 1], height / dim, "e4m3")


@pytest.mark.parametrize("lens,heads", [([37], 1), ([5, 300, 41], 2), ([37] * 60, 3)])
@pytest.mark.parametrize("q", [-1e31, -1e36])
def test_attention_of_very_low_scores(lens, heads, q):
    """Scores of -1e33 and -1e38, all equal: the mean of the values, also where most
    warps have no token."""
    dim = 128
    c = Cache(lens, heads, dim, 32, "e4m3", seed=55)
    c.k[:] = layer.e4m3.encode_rne_sat(np.float32(1))
    c.ks[:] = 1
    Q = np.full((len(lens), heads * 2, dim), q, np.float32)
    got, Qr = _attend(c, Q, None, 1.0, "e4m3")
    _check(got, c, Qr, _offsets([1] * len(lens)), 1.0, "e4m3")
    assert np.abs(got).min(axis=(1, 2)).max() > 0


@pytest.mark.parametrize("dim,group,block,fmt,q,what", [
    (*c, w) for c in ((128, 1, 16, "e4m3", 4), (64, 8, 32, "e5m2", 5), (128, 4, 64, "e4m3", 12),
                      (128, 16, 128, "e5m2", 3), (64, 1, 16, "e4m3", 40))
    for w in ("values", "keys", "infinite values", "scale") if c[3] == "e5m2" or w != "infinite values"])
@pytest.mark.parametrize("B", [1, 50])
def test_attention_hides_what_is_not_finite_from_those_before_it(dim, group, block, fmt, q, what, B):
    """A new token whose value, key or (first of a block) scale is not finite: the
    queries before it are what they are without it, those that see it are not finite."""
    heads, at = 2, q // 2  # the new token concerned
    n = 5 * block + q - at  # so that it begins a block
    clean = Cache([n] * B, heads, dim, block, fmt, seed=60)
    g = np.random.default_rng(61)
    Q = g.standard_normal((B * q, heads * group, dim)).astype(np.float32)
    want, Qr = _attend(clean, Q, None, dim ** -0.5, fmt)
    c = Cache([n] * B, heads, dim, block, fmt, seed=60)
    hit = [0, B // 2] if B > 1 else [0]
    for b_ in hit:
        blk = c.table[b_, 5]
        if what == "values":
            c.v[blk, 1, 0, ::3] = 0x7F if fmt == "e4m3" else 0x7E
        elif what == "infinite values":
            c.v[blk, 1, 0, ::3] = 0xFC
        elif what == "keys":
            c.k[blk, 1, 0] = 0x7F
        else:
            c.vs[blk, 1] = np.nan
    got, _ = _attend(c, Q, None, dim ** -0.5, fmt)
    got, want = (x.reshape(B, q, heads, group, dim) for x in (got, want))
    seen = np.zeros(got.shape, bool)
    seen[hit, at:, 1] = True
    if "values" in what:
        dims = np.arange(dim) % 3 == 0
        seen &= dims
    assert np.array_equal(got[~seen], want[~seen])
    assert not np.isfinite(got[seen]).any()
    if what != "infinite values":
        cu = _offsets([q] * B)
        O, _ = layer.kv_attention(Qr, c.k, c.ks, c.v, c.vs, c.table, c.lens, cu, dim ** -0.5, fmt)
        assert np.array_equal(np.isnan(O).reshape(got.shape), np.isnan(got))
