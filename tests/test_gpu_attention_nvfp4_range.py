"""Attention over the NVFP4 cache where keys and values lie far apart in size, against the float64
oracle on the values that the cache holds; the bounds are those of test_gpu_attention_nvfp4.py.

Both kernels (few query rows a sequence, and prompts), whole and cut into parts that are joined.
The sum of the weights, and so lse, must not depend on the values at all.
"""
import numpy as np
import pytest
import torch

from oracle import kvcache_nvfp4 as okv
from oracle.codecs import bf16_bits_to_f32, f32_to_bf16_bits_rne
from tests.helpers import DEV, bf16_bits_of, to_dev
from tests.test_gpu_attention_nvfp4 import Seqs

pytestmark = pytest.mark.gpu

ql = pytest.importorskip("quantized_linear_layers_block_amd")


def _bits(x):
    return f32_to_bf16_bits_rne(x.astype(np.float32))


def _rewrite(s, b, k, v):
    """Sequence b's keys and values [n, H, D]."""
    slots = torch.from_numpy(okv.sequence_slots(s.table[b], k.shape[0], s.page)).to(DEV)
    ql.kv_store_nvfp4(to_dev(_bits(k)), to_dev(_bits(v)), slots, s.cache)
    torch.cuda.synchronize()
    s.data = s.cache.data.cpu().numpy()


def _queries(s, q):
    s.q_bits = _bits(q)
    s.q = to_dev(s.q_bits)[:s.tq]


# log2 of the size of value row t of n (None: a zero row)
SPREADS = {
    "zero rows beside large ones": lambda t, n: None if t % 3 else 47,
    "zero rows, then large ones": lambda t, n: None if t < n // 2 else 50,
    "large rows, then zero ones": lambda t, n: 50 if t < n // 2 else None,
    "from the smallest to the largest": lambda t, n: -120 + 240 * t // n,
    "from the largest to the smallest": lambda t, n: 120 - 240 * t // n,
    "the ends of the range": lambda t, n: 125 if t % 16 == 3 else -95,
    "zero rows only": lambda t, n: None,
    "large rows only": lambda t, n: 120,
}


def _sized(g, n, h, d, size):
    v = g.standard_normal((n, h, d))
    for t in range(n):
        e = size(t, n)
        v[t] *= 0.0 if e is None else 2.0 ** e
    return v


@pytest.mark.parametrize("spread", SPREADS)
@pytest.mark.parametrize("nq,n,hq,h,d,logits", [
    (1, 90, 4, 2, 128, 0.0), (3, 200, 8, 1, 64, 1.0), (5, 333, 16, 8, 256, 0.3),   # few rows
    (1, 9000, 2, 1, 64, 0.5),                                                      # cut, joined by a kernel
    (150, 170, 2, 2, 128, 0.0), (140, 300, 2, 1, 64, 1.0), (200, 200, 1, 1, 256, 0.3),   # prompts
    (130, 2500, 2, 1, 128, 0.5)])                                                  # cut along the tokens
def test_the_sum_of_weights_does_not_depend_on_the_values(spread, nq, n, hq, h, d, logits):
    s = Seqs([(nq, n)], hq, h, d, 16, nq + d)
    g = np.random.default_rng(n)
    _rewrite(s, 0, g.standard_normal((n, h, d)) * logits, _sized(g, n, h, d, SPREADS[spread]))
    s.check(*s.run(), rows=8)


@pytest.mark.parametrize("spread", ["zero rows, then large ones", "from the largest to the smallest"])
def test_the_sum_of_weights_over_many_workgroups(spread):
    """Long sequences of some units that several workgroups share, joined by the last to arrive."""
    s = Seqs([(2, 6000), (2, 900)] * 2, 32, 4, 128, 64, 3)
    g = np.random.default_rng(5)
    for b, (_, n) in enumerate(s.lens):
        _rewrite(s, b, g.standard_normal((n, 4, 128)) * 0.4, _sized(g, n, 4, 128, SPREADS[spread]))
    s.check(*s.run(), rows=2, every=2)


@pytest.mark.parametrize("gap", [14, 19, 24, 28, 29, 33, 40, 70, 130])
@pytest.mark.parametrize("nq,n,hq,h,d", [(150, 160, 1, 1, 64), (140, 300, 2, 1, 128), (200, 200, 1, 1, 256),
                                         (130, 2500, 2, 1, 128), (3, 50, 2, 1, 128)])
def test_value_rows_far_apart_in_sixteen_tokens(gap, nq, n, hq, h, d):
    """A row 2^gap larger than the others of its 16 tokens; the queries before it see the others
    alone, and so do some behind it, which give it next to no weight."""
    s = Seqs([(nq, n)], hq, h, d, 16, gap)
    g = np.random.default_rng(gap)
    k, v = g.standard_normal((n, h, d)) * 0.3, g.standard_normal((n, h, d))
    q = g.standard_normal((max(s.tq, 1), hq, d))
    big = np.arange(5, n, 32)
    v[big] *= 2.0 ** min(gap, 120)
    v[big + 1 if big[-1] + 1 < n else big[:-1] + 1] *= 2.0 ** (min(gap, 120) - gap)
    k[..., 0], q[..., 0] = 0.0, 0.0
    k[big, :, 0] = -80.0                     # logits far below the others for the queries with a large element 0
    q[::2, :, 0] = 4.0 * d ** 0.5
    _rewrite(s, 0, k, v)
    _queries(s, q)
    s.check(*s.run(), rows=20)


@pytest.mark.parametrize("gap", [14, 18, 19, 24, 28, 29, 33, 40, 70])
@pytest.mark.parametrize("nq,n,hq,h,d", [(150, 160, 1, 1, 64), (140, 300, 2, 1, 128), (200, 200, 1, 1, 256),
                                         (130, 2500, 2, 1, 128), (3, 50, 2, 1, 128)])
def test_key_rows_far_apart_in_sixteen_tokens(gap, nq, n, hq, h, d):
    """Key rows 2^gap smaller than one of their 16, which lies across all queries (logit 0)."""
    s = Seqs([(nq, n)], hq, h, d, 16, gap)
    g = np.random.default_rng(gap)
    k, q = g.standard_normal((n, h, d)) * 2.0 ** -gap, g.standard_normal((max(s.tq, 1), hq, d)) * 2.0 ** gap
    q[..., :16] = 0.0
    k[5::16] = 0.0
    k[5::16, :, 3] = 4.0
    _rewrite(s, 0, k, g.standard_normal((n, h, d)))
    _queries(s, q)
    s.check(*s.run(), rows=20)


def test_prompt_rows_beside_a_nan_token():
    """Small values in the 16 tokens of a NaN token, which the checked queries do not see."""
    s = Seqs([(100, 160)], 2, 1, 128, 16, 8)
    g = np.random.default_rng(8)
    k, v = g.standard_normal((160, 1, 128)), g.standard_normal((160, 1, 128)) * 2.0 ** -40
    _rewrite(s, 0, k, v)
    bad = _bits(k[:1])
    bad[0, 0, 9] = 0x7FC0
    slot = torch.from_numpy(okv.sequence_slots(s.table[0], 160, 16)[140:141]).to(DEV)
    ql.kv_store_nvfp4(to_dev(bad), to_dev(_bits(v[:1])), slot, s.cache)
    out, lse = s.run()
    s.data = s.cache.data.cpu().numpy()
    assert torch.isnan(out[80:]).all() and torch.isnan(lse[80:]).all()
    s.check(out, lse, only=[0, 3, 60, 70, 75, 78, 79])


def _check_seen(s, out, lse, window, picks):
    """Query rows `picks` of the one sequence, with a bound that takes only what a row sees.  A weight's
    rounding below f16's smallest normal is at most 2^-25 against p = 2^(logit + F - m + 9) of the
    token that set m.  A token's share of out is p vhat 2^(ev - F + 4) 2^-13 2^m / sum 2^logit, with
    vhat 2^(ev - F + 4) <= 43008: so it is off by at most 2^-22.6 2^m / sum 2^logit.  m = logit + F of a token a
    that the row sees, F is at most 2^5 above the exponent of a's own row, and that row's largest value is 1260 2^ev
    or more: 2^(-22.6 + 5 - 10.3) = 2^-27.9 of the weight of a times its largest value, a token seen."""
    (nq, n), = s.lens
    qf = bf16_bits_to_f32(s.q_bits).astype(np.float64)
    o, z = bf16_bits_to_f32(bf16_bits_of(out)).astype(np.float64), lse.cpu().numpy().astype(np.float64)
    k, v = okv.load(s.data, okv.sequence_slots(s.table[0], n, s.page), s.d)
    for i in picks:
        hi = n - nq + i + 1
        lo = max(hi - window, 0) if window else 0
        ro, rz, am = okv.attention(qf[i][None], k[lo:hi], v[lo:hi], s.d ** -0.5)
        for j in range(s.hq):
            g = j // (s.hq // s.h)
            w = np.exp(s.d ** -0.5 * (k[lo:hi, g] @ qf[i, j]) - rz[0, j])
            share = (w * np.abs(v[lo:hi, g]).max(axis=1)).max()
            tol = 2.0 ** -8 * np.abs(ro[0, j]) + (2.0 ** -11 + 2.0 ** -12) * am[0, j] + (hi - lo) * 2.0 ** -27 * share + 1e-30
            err = np.abs(o[i, j] - ro[0, j])
            assert (err <= tol).all(), (i, j, err.max(), tol[err > tol].min())
            assert abs(z[i, j] - rz[0, j]) <= 2.0 ** -16 + 2.0 ** -20 * abs(rz[0, j])


@pytest.mark.parametrize("gap", [3, 5, 6, 10, 17, 18, 19, 27, 34, 60, 115])
@pytest.mark.parametrize("nq,n,hq,h,d", [(150, 160, 1, 1, 64), (140, 300, 2, 1, 128), (200, 200, 1, 1, 256),
                                         (130, 2500, 2, 1, 128), (3, 50, 2, 1, 128)])
@pytest.mark.parametrize("window", [0, 40])
def test_large_values_that_a_query_does_not_see(gap, nq, n, hq, h, d, window):
    """Value rows 2^gap larger than all others in the same 16 tokens as the last (or, with a window,
    the first) ones that a query sees; and seen ones that get no weight.  They must not take bits
    from the weights of the tokens in other groups."""
    s = Seqs([(nq, n)], hq, h, d, 16, gap)
    g = np.random.default_rng(gap)
    k, v, q = g.standard_normal((n, h, d)), g.standard_normal((n, h, d)), g.standard_normal((s.tq, hq, d))
    k[..., 0], q[..., 0] = 0.0, 12.0 * d ** 0.5
    first = n - nq + 20     # from here on seen by later queries only
    big = np.arange(first // 16 * 16 + 13, n, 48)
    v[big] *= 2.0 ** gap
    k[big, :, 0] = -20.0    # a logit of -240: no weight where they are seen
    _rewrite(s, 0, k, v)
    _queries(s, q)
    out, lse = s.run(window=window)
    near = [b - (n - nq) + x for b in big[:4] for x in (-13, -5, -1, 0, 1, window + 1, window + 3)]
    picks = sorted({i for i in near if 0 <= i < nq} | {0, nq // 2, nq - 1})
    _check_seen(s, out, lse, window, picks)


@pytest.mark.parametrize("gap", [3, 5, 6, 8, 12, 14, 16, 17, 22])
@pytest.mark.parametrize("nq,n,d", [(150, 1000, 64), (140, 1400, 128), (200, 1500, 256), (130, 4000, 128)])
@pytest.mark.parametrize("window", [0, 700])
def test_many_small_weights_behind_a_large_value_row_that_does_not_count(gap, nq, n, d, window):
    """One token with a weight of 2^10 in the 16 of the large row, and a thousand of weight 1 behind it
    that carry half of the output: all rounded alike, so that lost bits add up.  The large row is before the
    window, or has no weight."""
    s = Seqs([(nq, n)], 1, 1, d, 16, gap)
    g = np.random.default_rng(gap)
    first = n - nq + 45 - (window or n - nq)   # of the tokens that query 44 sees through the window
    big = (first + 15) // 16 * 16 + 3
    i0 = 44 + big - first + 1                  # the first query that does not see it
    k, q = np.zeros((n, 1, d)), np.zeros((s.tq, 1, d))
    q[:, 0, 1] = d ** 0.5 * (1 + g.integers(0, 8, s.tq) / 64)
    q[:, 0, 2] = d ** 0.5
    k[big + 8, 0, 1] = 7.0
    k[big, 0, 2] = 0.0 if window else -200.0
    v = 1 + 0.1 * g.standard_normal((n, 1, d))
    v[big + 8] *= -1
    v[big] = 1.6 * 2.0 ** gap
    _rewrite(s, 0, k, v)
    _queries(s, q)
    out, lse = s.run(window=window)
    _check_seen(s, out, lse, window, range(i0, i0 + 8))


# (log2 of the queries, of the keys that meet them, of the ones that lie across them, softmax scale)
ENDS = {"large queries, small keys": (100, -98, 120, 0.125), "small queries, large keys": (-131, 124, -120, 3.0),
        "large both, across": (120, -119, 126, 0.3), "a large scale": (-60, -50, 0, 2.0 ** 108),
        "a small scale": (70, 50, 40, 2.0 ** -119), "a small negative scale": (70, 50, 40, -2.0 ** -119),
        "the smallest queries": (-133, 127, 100, 16.0)}


@pytest.mark.parametrize("ends", ENDS)
@pytest.mark.parametrize("nq,n,hq,h,d", [(1, 60, 4, 2, 128), (3, 200, 8, 1, 64), (5, 333, 16, 8, 256), (1, 9000, 2, 1, 64),
                                         (150, 170, 2, 2, 128), (140, 300, 2, 1, 64), (200, 200, 1, 1, 256),
                                         (130, 2500, 2, 1, 128)])
def test_queries_and_keys_at_the_ends_of_their_range(ends, nq, n, hq, h, d):
    """Products of ordinary size of factors that float32 cannot hold the scales of, beside keys
    that a query is at right angles to (logit 0)."""
    eq, ek, across, scale = ENDS[ends]
    s = Seqs([(nq, n)], hq, h, d, 16, nq + d)
    g = np.random.default_rng(n)
    # (queries of one binade and few bits: the smallest bf16 hold them exactly)
    q = (1 + g.integers(0, 2, (s.tq, hq, d)) / 2) * g.choice([-1.0, 1.0], (s.tq, hq, d))
    k = g.standard_normal((n, h, d)) * 0.3
    k[..., :16], q[..., :16] = 0.0, 0.0
    q[..., 16:24] = 1.0
    k[3::7] = 0.0
    q, k = np.ldexp(q, eq), np.ldexp(k, ek)
    k[3::7, :, 5] = 2.0 ** across
    _rewrite(s, 0, k, g.standard_normal((n, h, d)))
    _queries(s, q)
    s.check(*s.run(softmax_scale=scale), scale=scale, rows=8)


@pytest.mark.parametrize("nq,n,d", [(1, 60, 128), (3, 200, 64), (2, 9000, 64), (150, 170, 128), (130, 2500, 64), (200, 200, 256)])
@pytest.mark.parametrize("eq,ek", [(100, 60), (20, 118)])
def test_logits_beyond_float32(nq, n, d, eq, ek):
    """A key whose logit is below float32 has no weight and changes nothing else; one whose logit is above it
    gives the queries that see it NaN, and no others."""
    s = Seqs([(nq, n)], 1, 1, d, 16, nq + d)
    g = np.random.default_rng(n)
    q, k = np.zeros((s.tq, 1, d)), np.zeros((n, 1, d))
    q[..., :4], q[..., 16:] = 2.0 ** eq, 2.0 ** eq * g.choice([-1.0, 1.0], (s.tq, 1, d - 16))
    k[..., 16:] = g.standard_normal((n, 1, d - 16)) * 2.0 ** -eq
    low, high = 5, n - 3
    k[low] = 0.0
    k[low, 0, 2] = -2.0 ** ek
    v = g.standard_normal((n, 1, d))
    _rewrite(s, 0, k, v)
    _queries(s, q)
    s.check(*s.run(softmax_scale=1.0), scale=1.0, rows=12)
    k[high] = 0.0
    k[high, 0, 1] = 2.0 ** ek
    _rewrite(s, 0, k, v)
    out, lse = s.run(softmax_scale=1.0)
    first = max(high - (n - nq), 0)
    assert torch.isnan(out[first:]).all() and torch.isnan(lse[first:]).all()
    if first:
        s.check(out, lse, scale=1.0, only=sorted({0, first // 2, first - 1}))
