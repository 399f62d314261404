"""fp8_kv_attention_chunk within its rounding, against the FP64 oracle.

Bound, derived before the first run (that of fp8_kv_attention): p is rounded to FP16 (2^-11
relative, or 2^-25 of the row's largest term absolute), scores, exponentials and sums are FP32
(together under 2^-12 relative here), the output BF16 (2^-8 of the value):
  |got - ref| <= 2^-8 |ref| + 2^-10 sum p |v| + n 2^-24 max |v|
"""

import numpy as np
import pytest

from oracle import layer
from tests.gpu_helpers import dev, host
from tests.test_gpu_kv import _CODES, Cache, _offsets

pytestmark = pytest.mark.gpu


def _queries(T, hq, dim, seed, size=2.0):
    return (size * np.random.default_rng(seed).standard_normal((T, hq, dim))).astype(np.float32)


def _run(c, Q, counts, scale=None, causal=True, max_q=None, fmt=None):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    tQ = dev(Q).to(torch.bfloat16)
    O = torch.full(tQ.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    cu = _offsets(counts)
    b.fp8_kv_attention_chunk(tQ, *c.on_gpu(), cu_q=dev(cu), max_q=max(counts) if max_q is None else max_q, scale=scale,
                             causal=causal, fmt=c.fmt, O=O)
    return O, tQ.double().cpu().numpy(), cu


def _check(O, c, Q, cu, scale=None, causal=True):
    dim = Q.shape[2]
    ref, A = layer.kv_attention_chunk(Q, c.k, c.ks, c.v, c.vs, c.table, c.lens, cu, dim ** -0.5 if scale is None else scale,
                                      c.fmt, causal)
    got = host(O)
    none = np.isnan(ref)
    assert np.isnan(got[none]).all()  # rows of no sequence stay
    vmax = np.nanmax(np.abs(np.where(np.isfinite(x := _CODES[c.fmt].decode(c.v)), x, 0)) * c.vs[:, :, None, None].astype(np.float64))
    bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * A + max(c.lens.max(), 1) * 2.0 ** -24 * vmax
    bad = ~(np.abs(got - ref) <= bound) & ~none
    assert not bad.any(), (int(bad.sum()), bad.size, got[bad][:4], ref[bad][:4], np.argwhere(bad)[:4])


CASES = [  # cached tokens (new ones included), new tokens, heads, group, dim, block, format
    ([1], [1], 1, 1, 64, 16, "e4m3"), ([17], [17], 2, 1, 64, 16, "e4m3"), ([54], [17], 2, 1, 64, 16, "e5m2"),
    ([128], [128], 1, 1, 128, 64, "e4m3"), ([129], [129], 1, 2, 128, 128, "e4m3"), ([300], [300], 2, 4, 128, 64, "e4m3"),
    ([0, 5, 300, 16], [0, 5, 100, 1], 2, 3, 128, 32, "e4m3"), ([600, 601, 3], [257, 1, 3], 1, 8, 128, 16, "e5m2"),
    ([1000, 17, 640], [60, 17, 513], 2, 5, 64, 128, "e4m3"), ([4099], [2], 2, 8, 128, 64, "e4m3"),
    ([2, 5], [4, 6], 1, 2, 64, 16, "e4m3"),  # more queries than tokens: the first see none
    ([33] * 70, [3] * 70, 2, 2, 64, 16, "e4m3"), ([2000], [700], 1, 1, 64, 32, "e5m2"), ([513], [513], 3, 7, 128, 32, "e4m3")]


@pytest.mark.parametrize("lens,counts,heads,group,dim,block,fmt", CASES)
@pytest.mark.parametrize("causal", [True, False])
def test_attention(lens, counts, heads, group, dim, block, fmt, causal):
    from fp8_fine_grained_e4m3_gb300 import binding as b
    c = Cache(lens, heads, dim, block, fmt, seed=sum(lens)).stale()
    O, Q, cu = _run(c, _queries(sum(counts), heads * group, dim, 7), counts, causal=causal)
    _check(O, c, Q, cu, causal=causal)
    assert b.fp8gemm_get_device_status() == b.OK


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_blocks_and_formats(block, dim, fmt):
    c = Cache([777, 130, 64], 2, dim, block, fmt, seed=block + dim).stale()
    counts = [200, 130, 1]
    O, Q, cu = _run(c, _queries(sum(counts), 4, dim, block), counts)
    _check(O, c, Q, cu)


def test_equal_counts_without_offsets_and_parts_of_fused_rows():
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    heads, group, dim, B, n = 2, 4, 128, 3, 50
    c = Cache([70, 50, 300], heads, dim, 32, "e4m3", seed=5).stale()
    w = heads * group * dim
    qkv = dev(np.random.default_rng(6).standard_normal((B * n, w + 2 * heads * dim)).astype(np.float32)).to(torch.bfloat16)
    tQ = qkv[:, :w].unflatten(1, (heads * group, dim))
    O = b.fp8_kv_attention_chunk(tQ, *c.on_gpu(), scale=0.1)
    _check(O, c, tQ.double().cpu().numpy(), _offsets([n] * B), 0.1)


def test_rows_behind_the_last_sequence_stay():
    c = Cache([100, 60], 2, 64, 16, "e4m3", seed=8)
    O, Q, cu = _run(c, _queries(80, 4, 64, 1), [30, 40])
    _check(O, c, Q, cu)
    assert np.isnan(host(O)[70:]).all()


@pytest.mark.parametrize("kind", ["peaked", "flat", "rising", "falling", "tiny_q", "huge_q", "wide_scales", "wide_values",
                                  "zero_scales", "negative_scales", "mixed_rows"])
def test_statistics(kind):
    """Scores that one token dominates, all equal, rising or falling along the cache, queries near the ends of
    BF16's range, rows of very different sizes, and scales of neighbouring blocks that differ by 2^40 or are 0."""
    heads, dim, n, new = 1, 128, 700, 150
    c = Cache([n], heads, dim, 16, "e4m3", seed=9, spread=20 if kind == "wide_values" else 1)
    g = np.random.default_rng(10)
    Q = g.standard_normal((new, 2, dim)).astype(np.float32)
    scale = dim ** -0.5
    enc = layer.e4m3.encode_rne_sat
    if kind == "peaked":
        c.k[c.table[0, 20], 0, 3] = enc((50 * np.sign(Q[0, 0])).astype(np.float32))
        Q[:] = Q[:1, :1]
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
        c.ks[:] = (2.0 ** g.integers(-40, -5, c.ks.shape)).astype(np.float32)
    elif kind == "wide_values":
        c.ks[:] = 2.0 ** -6
    elif kind == "zero_scales":
        c.vs[::3], c.ks[1::3] = 0, 0
    elif kind == "negative_scales":
        c.vs[::2] *= -1
        c.ks[1::3] *= -1.25
    elif kind == "mixed_rows":
        Q *= np.exp2(g.integers(-60, 3, (new, 2, 1))).astype(np.float32)
    O, Qr, cu = _run(c, Q, [new], scale=scale)
    _check(O, c, Qr, cu, scale)


def test_small_values_beside_large_ones_that_are_hidden():
    """Value scales of 2^-40 in the tokens that the first queries see, 1 in those that they do not: each query
    keeps the precision of what it sees."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    dim, n, new = 64, 256, 200
    c = Cache([n], 1, dim, 16, "e4m3", seed=20, spread=0)
    for j in range(c.width):
        c.vs[c.table[0, j]] = 2.0 ** -40 if j < 8 else 1.0
    O, Q, cu = _run(c, _queries(new, 2, dim, 21), [new])
    ref, A = layer.kv_attention_chunk(Q, c.k, c.ks, c.v, c.vs, c.table, c.lens, cu, dim ** -0.5)
    sees = n - new + 1 + np.arange(new)
    got = host(O)
    first = sees <= 128
    assert np.all(np.abs(got - ref)[first] <= (2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * A + n * 2.0 ** -24 * 448 * 2.0 ** -40)[first])
    _check(O, c, Q, cu)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("what", ["key", "value", "key scale", "value scale"])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_what_is_not_finite_reaches_only_the_queries_that_see_it(fmt, what, bad):
    """A key, value or scale that is not finite, in a token that the last queries alone see."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    dim, n, new, at = 64, 400, 300, 333
    c = Cache([n], 2, dim, 16, fmt, seed=30)
    blk, off = c.table[0, at // 16], at % 16
    clean, Q, cu = _run(c, _queries(new, 4, dim, 31), [new])
    code = 0x7f if fmt == "e4m3" or np.isnan(bad) else 0x7c
    if what == "key":
        c.k[blk, 1, off, 5] = code
    elif what == "value":
        c.v[blk, 1, off, 5] = code
    else:
        (c.ks if what == "key scale" else c.vs)[blk, 1] = bad
        at = at // 16 * 16
    O, _, _ = _run(c, _queries(new, 4, dim, 31), [new])
    got, ok = host(O), host(clean)
    sees = n - new + 1 + np.arange(new)
    hit = sees > at
    assert np.array_equal(got[~hit], ok[~hit]) and np.array_equal(got[:, :2], ok[:, :2])
    touched = got[hit][:, 2:]
    if what == "value":
        assert not np.isfinite(touched[..., 5]).any()
        assert np.array_equal(np.delete(touched, 5, 2), np.delete(ok[hit][:, 2:], 5, 2))
    elif what == "value scale":
        assert not np.isfinite(touched).any()
    else:
        # a score of -infinity has weight 0 and leaves the row finite; one of +infinity or NaN does not
        # (scores are the products of query and codes, times the scale)
        with np.errstate(all="ignore"):
            x = np.einsum("nhd,ld->nhl", Q[hit][:, 2:], layer._FORMATS[fmt][2](c.k[blk, 1])) * np.float64(c.ks[blk, 1])
        there = np.arange(at // 16 * 16, at // 16 * 16 + 16) < sees[hit][:, None]
        lost = (there[:, None] & ~(x < np.inf)).any(2)
        assert np.array_equal(np.isfinite(touched).all(2), ~lost) and np.array_equal(np.isnan(touched).all(2), lost)


def test_bad_tables_and_lengths_set_the_status():
    from fp8_fine_grained_e4m3_gb300 import binding as b
    c = Cache([200, 100], 1, 64, 16, "e4m3", seed=40).stale()
    good = c.table.copy()
    for entry in (-1, c.n, 2 ** 31 - 1, -2 ** 31):
        c.table = good.copy()
        c.table[0, 3] = entry
        O, Q, cu = _run(c, _queries(150, 2, 64, 41), [100, 50])
        assert b.fp8gemm_get_device_status() == b.ERR_DEVICE_STATUS
        # the tokens of that block are not there: as if their scores were -infinity
        c.table = good
        k, v = c.k.copy(), c.v.copy()
        ref = np.zeros(Q.shape)
        for i in range(100):
            sees = 101 + i
            j = np.array([x for x in range(sees) if x // 16 != 3])
            for h in range(2):
                kk, vv = (np.stack([layer.e4m3.decode(a[good[0, x // 16], 0, x % 16]) * np.float64(s[good[0, x // 16], 0])
                                    for x in j]) for a, s in ((k, c.ks), (v, c.vs)))
                x = kk @ Q[i, h] / 8
                p = np.exp(x - x.max())
                ref[i, h] = p @ vv / p.sum()
        assert np.abs(host(O)[:100] - ref[:100]).max() <= 2.0 ** -6 * np.abs(ref).max()
    for lens in ([-1, 100], [16 * c.width + 1, 100]):
        c.lens = np.array(lens, np.int32)
        O, Q, cu = _run(c, _queries(150, 2, 64, 41), [100, 50])
        assert b.fp8gemm_get_device_status() == b.ERR_DEVICE_STATUS
        assert not host(O)[:100].any() and np.isfinite(host(O)[100:]).all()
    c.lens = np.array([200, 100], np.int32)
    O, Q, cu = _run(c, _queries(150, 2, 64, 41), [100, 50], max_q=60)  # a sequence with more than it may have
    assert b.fp8gemm_get_device_status() == b.ERR_DEVICE_STATUS
    assert np.isnan(host(O)[:100]).all() and np.isfinite(host(O)[100:]).all()
    assert b.fp8gemm_get_device_status() == b.OK


def test_long_cache_past_32_bit_offsets():
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    heads, dim, block = 8, 128, 128
    n = 2 ** 32 // (heads * dim * block) + 40
    c = Cache([1500], heads, dim, block, "e4m3", seed=12, spare=0)
    k, v = (torch.zeros((n, heads, block, dim), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((n, heads), device="cuda") for _ in range(2))
    far = n - c.n
    k[far:], v[far:], ks[far:], vs[far:] = dev(c.k), dev(c.v), dev(c.ks), dev(c.vs)
    tQ = dev(_queries(40, heads * 2, dim, 3)).to(torch.bfloat16)
    O = b.fp8_kv_attention_chunk(tQ, k, ks, v, vs, dev(c.table) + far, dev(c.lens))
    _check(O, c, tQ.double().cpu().numpy(), [0, 40])


def test_same_as_single_tokens():
    """The chunk's last queries beside fp8_kv_attention's: each within its own bound."""
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    c = Cache([900, 33], 2, 128, 64, "e4m3", seed=50).stale()
    Q = dev(_queries(8, 8, 128, 51)).to(torch.bfloat16)
    one, many = b.fp8_kv_attention(Q, *c.on_gpu()), b.fp8_kv_attention_chunk(Q, *c.on_gpu())
    _check(many, c, Q.double().cpu().numpy(), [0, 4, 8])
    _check(one, c, Q.double().cpu().numpy(), [0, 4, 8])


def test_same_bits_on_every_run_in_a_graph_and_after_larger_calls():
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    small = Cache([3000], 2, 128, 64, "e4m3", seed=60)
    large = Cache([5000, 2000], 4, 128, 64, "e4m3", seed=61)
    ts, tl = small.on_gpu(), large.on_gpu()
    qs, ql = dev(_queries(20, 8, 128, 1)).to(torch.bfloat16), dev(_queries(800, 16, 128, 2)).to(torch.bfloat16)
    want = b.fp8_kv_attention_chunk(qs, *ts)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        b.fp8_kv_attention_chunk(qs, *ts)
        s.synchronize()
        held = b.workspace_bytes()
        graph, got = torch.cuda.CUDAGraph(), torch.empty_like(want)
        with torch.cuda.graph(graph, stream=s):
            b.fp8_kv_attention_chunk(qs, *ts, O=got)
        b.fp8_kv_attention_chunk(ql, *tl)
        s.synchronize()
        assert b.workspace_bytes() == held
        for _ in range(3):
            got.zero_()
            graph.replay()
            s.synchronize()
            assert torch.equal(got, want)
        ts[5].fill_(2500)  # a replay with another length
        graph.replay()
        s.synchronize()
        assert torch.equal(got, b.fp8_kv_attention_chunk(qs, *ts))
    b.fp8gemm_release_workspaces(s)
    assert b.fp8gemm_get_device_status() == b.OK


@pytest.mark.parametrize("n,heads,tiles,launches", [(100, 2, 4, 1), (100, 2, 5, 2), (700, 32, 8, 1), (700, 32, 9, 2), (700, 8, 8, 2)])
def test_units_whole_or_split(n, heads, tiles, launches):
    """By the table's width and the units: the same results."""
    from fp8_fine_grained_e4m3_gb300 import binding as b
    c = Cache([n], heads, 64, 128, "e4m3", seed=tiles).stale()
    c.table = np.concatenate([c.table, np.zeros((1, tiles), c.table.dtype)], 1)[:, :tiles]
    c.width = tiles
    before = b.num_kernel_launches()
    O, Q, cu = _run(c, _queries(n, heads, 64, 3), [n])
    assert b.num_kernel_launches() - before == launches
    _check(O, c, Q, cu)


@pytest.mark.parametrize("lens,counts,heads,group,causal", [
    ([300], [4], 2, 8, True), ([300], [11], 2, 3, True),  # 32 rows and 33
    ([300, 2000], [1, 1], 2, 8, False), ([300, 2000], [2, 1], 2, 8, False),
    ([40 + i for i in range(64)], [1 + i % 2 for i in range(64)], 2, 8, True), ([9] * 64, [1] * 64, 2, 8, True)])
def test_few_rows(lens, counts, heads, group, causal):
    from fp8_fine_grained_e4m3_gb300 import binding as b
    c = Cache(lens, heads, 128, 16, "e4m3", seed=21).stale()
    O, Q, cu = _run(c, _queries(sum(counts), heads * group, 128, 22), counts, causal=causal)
    _check(O, c, Q, cu, causal=causal)
    wide, _, _ = _run(c, _queries(sum(counts), heads * group, 128, 22), counts, causal=causal, max_q=sum(counts) + 40)
    _check(wide, c, Q, cu, causal=causal)
    assert b.fp8gemm_get_device_status() == b.OK


def test_padded_batch_and_rows_of_one_warp():
    # empty sequences before, between and behind the others, in runs longer than a warp; causal rows whose warps see
    # ever more of a tile, one of them with a single row
    counts = [0] * 40 + [1] + [0] * 33 + [130] + [0] * 64 + [33, 0, 257] + [0] * 35
    lens = [0 if n == 0 else n + 3 * n % 50 for n in counts]
    c = Cache(lens, 3, 64, 32, "e4m3", seed=12).stale()
    for group in (1, 3):
        O, Q, cu = _run(c, _queries(sum(counts), 3 * group, 64, group), counts)
        _check(O, c, Q, cu)


@pytest.mark.parametrize("first", [(300, 1), (1, 300)])
def test_any_first_call_prepares_a_capture_of_few_or_many_rows(first):
    import torch
    from fp8_fine_grained_e4m3_gb300 import binding as b
    s = torch.cuda.Stream()
    for i, n in enumerate(first):
        c = Cache([400], 2, 128, 64, "e4m3", seed=n).stale()
        cache = c.on_gpu()
        Q = dev(_queries(n, 2, 128, n)).to(torch.bfloat16)
        O = torch.zeros_like(Q)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            if i == 0:
                b.fp8_kv_attention_chunk(Q, *cache, O=O)
                continue
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                b.fp8_kv_attention_chunk(Q, *cache, O=O)
            for _ in range(2):
                O.zero_()
                graph.replay()
            s.synchronize()
        _check(O, c, Q.double().cpu().numpy(), _offsets([n]))
    with torch.cuda.stream(s):
        assert b.fp8gemm_get_device_status() == b.OK
        b.fp8gemm_release_workspaces()
