"""fp8_kv_attention_chunk where the scores of a row rise far, and where scales, values and queries leave the ordinary range.

Weights are kept relative to the row's largest sum of 16 neighbouring terms p |v_scale|.  Bounds, derived before the
first run (the terms P of that sum, the numerators in FP16, are at least 2^5 together, and move in steps of 2^-24 at the
least, so a term is off by 2^-11 of itself or by 2^-30 of the sum, times its code; scores, exponentials and sums are
FP32, together under 2^-11 relative; the output is BF16):
  |got - ref| <= 2^-8 |ref| + 2^-10 sum p |v| + 2^-30 max over 16 (sum p |v_scale|) sum |code|
"""

import math

import numpy as np
import pytest

from oracle import layer
from tests.gpu_helpers import dev, host
from tests.test_gpu_chunk import _check, _queries, _run
from tests.test_gpu_kv import _CODES, Cache

pytestmark = pytest.mark.gpu

ONE = {"e4m3": 0x38, "e5m2": 0x3C}


def _cache(scores, dim=64, n=None, fmt="e4m3", seed=0):
    """One sequence and one head in blocks of 16: a query (x, 0, 0, ...) has the score x scores[j], in powers of two, with
    all tokens of block j.  Values are positive, their scales 2^-6."""
    c = Cache([16 * len(scores) if n is None else n], 1, dim, 16, fmt, seed=seed, spread=0)
    c.k[:] = 0
    c.k[..., 0] = ONE[fmt]
    for j, s in enumerate(scores):
        c.ks[c.table[0, j]] = s
    c.v &= 0x7F
    c.vs[:] = 2.0 ** -6
    return c


def _queries_of(sizes, dim=64):
    Q = np.zeros((len(sizes), 1, dim), np.float32)
    Q[:, 0, 0] = sizes
    return Q


def _within(O, c, Q, cu, causal, dims=slice(None), scale=math.log(2)):
    """The bound above, for one sequence and one head."""
    ref, A = layer.kv_attention_chunk(Q, c.k, c.ks, c.v, c.vs, c.table, c.lens, cu, scale, c.fmt, causal)
    n, new = int(c.lens[0]), len(Q)
    blocks = c.table[0, :-(-n // 16)]
    k = np.concatenate([_CODES[c.fmt].decode(c.k[x, 0]) * np.float64(c.ks[x, 0]) for x in blocks])[:n]
    vs = np.repeat(np.abs(c.vs[blocks, 0].astype(np.float64)), 16)[:n]
    sees = n - new + 1 + np.arange(new) if causal else np.full(new, n)
    x = np.where(np.arange(n) < sees[:, None], scale * (Q[:, 0].astype(np.float64) @ k.T), -np.inf)
    p = np.exp(x - x.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    codes = np.abs(np.concatenate([_CODES[c.fmt].decode(c.v[x, 0]) for x in blocks])[:n])
    top = np.add.reduceat(p * vs, np.arange(0, n, 16), 1).max(1)
    floor = 2.0 ** -30 * top[:, None] * (np.arange(n) < sees[:, None]) @ codes
    err = np.abs(host(O) - ref)
    ok = err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * A + floor[:, None]
    assert ok[..., dims].all(), (float((err / (np.abs(ref) + 1e-300))[..., dims].max()), np.argwhere(~ok)[:4])


@pytest.mark.parametrize("causal", [True, False])
def test_rows_of_one_warp_of_which_some_rise_further(causal):
    """In a tile that some row does not see whole, every second row's scores rise by 2^20 and the others' by 2^7.5: each
    row's reference is its own."""
    c = _cache([0] * 8 + [20] + [0] * 4, n=200)
    O, Q, cu = _run(c, _queries_of([0.375 if i % 2 else 1.0 for i in range(40)]), [40], scale=math.log(2), causal=causal)
    _check(O, c, Q, cu, math.log(2), causal)
    _within(O, c, Q, cu, causal)


@pytest.mark.parametrize("rise", [15.0, 18.3, 21.5, 23.4, 24.9, 25.2, 27.5, 30.0])
@pytest.mark.parametrize("causal,new", [(True, 40), (True, 300), (False, 40)])
def test_a_peak_in_the_last_tokens_of_a_masked_tile(rise, causal, new):
    """A tile that all rows see, then 96 tokens 2^9.9 above it and one token 2^rise above it whose values are 0 in half of
    the dimensions: those show what is left of the others' weights."""
    lead = 24 if new == 300 else 8  # whole tiles before
    c = _cache([0] * lead + [9.9] * 6 + [rise, 0], n=16 * lead + 122)
    peak = c.table[0, lead + 6]
    c.k[peak, 0, 1:] = 0
    c.v[peak, 0, 0, :32] = 0
    O, Q, cu = _run(c, _queries_of([1.0] * new), [new], scale=math.log(2), causal=causal)
    _check(O, c, Q, cu, math.log(2), causal)
    _within(O, c, Q, cu, causal)


def test_few_rows_leave_the_rows_behind_the_last_sequence():
    """Single tokens of a padded batch, which go to the kernel for few rows."""
    c = Cache([300, 0, 41, 7], 2, 64, 16, "e4m3", seed=95).stale()
    O, Q, cu = _run(c, _queries(9, 4, 64, 96), [1, 0, 2, 1])
    _check(O, c, Q, cu)
    assert np.isnan(host(O)[4:]).all()


@pytest.mark.parametrize("heads,group,counts,causal", [(1, 300, [3, 1], True), (2, 257, [2, 5], False), (1, 1000, [1, 1], True)])
def test_groups_wider_than_a_unit_of_rows(heads, group, counts, causal):
    c = Cache([140, 77], heads, 64, 32, "e4m3", seed=97).stale()
    O, Q, cu = _run(c, _queries(sum(counts), heads * group, 64, 98), counts, causal=causal)
    _check(O, c, Q, cu, causal=causal)


@pytest.mark.parametrize("rise", [11.3, 17.9, 21.7, 24.9])
@pytest.mark.parametrize("causal", [True, False])
def test_sixteen_equal_peaks_in_a_tile_that_all_rows_see(rise, causal):
    """What comes behind a peak of 16 equal tokens, in the same unit of four tiles: weights that lie half-way between
    two numbers of the fewest bits."""
    c = _cache([0] * 8 + [rise] + [-0.476] * 23)
    c.v[c.table[0, 8], 0, :, :32] = 0
    O, Q, cu = _run(c, _queries_of([1.0] * 40), [40], scale=math.log(2), causal=causal)
    _within(O, c, Q, cu, causal)


@pytest.mark.parametrize("power", [50, 20, -9, -25, -32, -40])
@pytest.mark.parametrize("causal", [True, False])
def test_blocks_of_zero_scale_beside_small_values(power, causal):
    """Blocks of zeros have the scale 0: they are in the sum of the weights and do not cost the others bits."""
    dim, n, new = 128, 700, 150
    c = Cache([n], 1, dim, 16, "e4m3", seed=70)
    c.vs[:] = 2.0 ** power
    c.vs[c.table[0, ::3]] = 0
    O, Q, cu = _run(c, _queries(new, 1, dim, 71), [new], causal=causal)
    _within(O, c, Q, cu, causal, scale=dim ** -0.5)
    c.vs[:] = 0
    O, Q, cu = _run(c, _queries(new, 1, dim, 71), [new], causal=causal)
    assert not host(O).any()


@pytest.mark.parametrize("rise", [12.0, 20.3, 25.0, 33.0])
@pytest.mark.parametrize("at", [0, 9, 17])
@pytest.mark.parametrize("causal", [True, False])
def test_a_block_of_zero_scale_that_dominates(rise, at, causal):
    """Zeros that the scores point to leave the rest of the output small, not rough: the bound is of the rest alone."""
    scores = [0] * 20
    scores[at] = rise
    c = _cache(scores, n=310)
    c.vs[c.table[0, at]] = 0
    O, Q, cu = _run(c, _queries_of([1.0] * 33), [33], scale=math.log(2), causal=causal)
    _within(O, c, Q, cu, causal)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -130])
@pytest.mark.parametrize("at", [40, 433])
@pytest.mark.parametrize("second", [False, True])
def test_what_is_not_finite_under_a_scale_of_zero(fmt, size, at, second):
    """0 times NaN is NaN, in a tile that all rows see and in one that some do not, whatever other tokens hold."""
    dim, n, new = 64, 600, 300
    c = Cache([n], 1, dim, 16, fmt, seed=80)
    c.vs[c.table[0, at // 16]] = size
    clean, Q, cu = _run(c, _queries(new, 2, dim, 81), [new])
    c.v[c.table[0, at // 16], 0, at % 16, 5] = 0x7F
    if second:
        c.v[c.table[0, 520 // 16], 0, 520 % 16, 9] = 0x7F
    O, _, _ = _run(c, _queries(new, 2, dim, 81), [new])
    sees = n - new + 1 + np.arange(new)
    want = host(clean).copy()
    want[sees > at, :, 5] = np.nan
    if second:
        want[sees > 520, :, 9] = np.nan
    assert np.array_equal(host(O), want, equal_nan=True)


@pytest.mark.parametrize("power", [-114, -116, -117, -120, -128])
def test_queries_near_the_least_of_their_type(power):
    """Queries of BF16's last normal numbers and below them, under key scales that make ordinary scores of them."""
    dim, n, new = 64, 300, 60
    c = Cache([n], 1, dim, 16, "e4m3", seed=90)
    c.ks = (c.ks * 2.0 ** 110).astype(np.float32)
    Q = _queries(new, 1, dim, 91) * np.float32(2.0 ** power)
    O, Qr, cu = _run(c, Q, [new], scale=dim ** -0.5 * 2.0 ** (-power - 110))
    _check(O, c, Qr, cu, dim ** -0.5 * 2.0 ** (-power - 110))
