"""The oracle of the NVFP4 KV cache against its definition: row exponents, rounding of codes by
exhaustive search, exact values, the layout as a bijection, NaN tokens and attention on cases
with a closed form."""
import numpy as np
import pytest

from oracle import kvcache_nvfp4 as okv
from oracle.codecs import bf16_bits_to_f32, e2m1_decode, e4m3_decode, f32_to_bf16_bits_rne


def _bits(x):
    return f32_to_bf16_bits_rne(np.asarray(x, np.float32))


def test_row_exponents():
    for amax, e in [(2688.0, 0), (2704.0, 1), (1344.0, -1), (1.0, -11), (1.3125, -11), (1.3203125, -10), (0.0, -100),
                    (2.0 ** -120, -100), (3.3895313892515355e38, 117)]:
        x = np.zeros((1, 64), np.float32)
        x[0, 5] = -amax
        assert okv.encode_rows(_bits(x))[2][0] == e, amax


@pytest.mark.parametrize("d", [64, 128, 256])
def test_codes_are_nearest_and_values_exact_in_bf16(d):
    g = np.random.default_rng(d)
    x = g.standard_t(3, size=(40, d)) * np.exp2(g.integers(-60, 60, size=(40, 1)))
    x[3] = 0
    bits = _bits(x)
    xf = bf16_bits_to_f32(bits).astype(np.float64)
    code, scale, e = okv.encode_rows(bits)
    unit = np.repeat(e4m3_decode(scale), 16, axis=1) * np.exp2(e.astype(np.float64))[:, None]
    val = e2m1_decode(code) * unit
    assert np.array_equal(bf16_bits_to_f32(_bits(val)).astype(np.float64), val)
    grid = e2m1_decode(np.arange(8, dtype=np.uint8))
    best = np.abs(np.abs(xf)[..., None] - grid * unit[..., None]).min(axis=-1)
    assert np.array_equal(np.abs(xf - val), best)
    # block scales use the range: the block with the row's maximum is within a step of 224..448
    top = e4m3_decode(scale).max(axis=1)
    assert ((top >= 216) | (np.abs(xf).max(axis=1) == 0)).all()


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (256, 32)])
def test_layout_is_a_bijection(d, page):
    data = okv.empty(3, 2, d, page)
    seen = np.zeros(data.size, int)
    for s in range(3 * page):
        for h in range(2):
            for a in okv._addresses(data, s, h, d):
                seen[a] += 1
    assert (seen == 1).all()


def test_store_load_round_trip_and_nan_tokens():
    g = np.random.default_rng(0)
    k, v = (_bits(g.standard_normal((6, 3, 64))) for _ in range(2))
    v[2, 1, 7] = 0x7F80
    k[4, 0, 0] = 0xFFC1
    data = okv.empty(2, 3, 64, 16, fill=0xEE)
    okv.store(data, k, v, [3, 17, 0, 31, 9, 32])   # 32: outside
    lk, lv = okv.load(data, [3, 17, 0, 31, 9, 32], 64)
    assert np.isnan(lk[2, 1]).all() and np.isnan(lv[2, 1]).all() and np.isnan(lk[4, 0]).all()
    assert np.isfinite(lk[2, 0]).all() and not lk[5].any()
    kf = bf16_bits_to_f32(k[0]).astype(np.float64)
    assert np.abs(lk[0] - kf).max() <= np.abs(kf).max() * (1 / 6 + 1 / 14)   # half the widest step, the scale's rounding
    assert (data.reshape(2, 3, -1) == 0xEE).sum() > 0
    # what is held stores as itself
    again = okv.empty(2, 3, 64, 16)
    okv.store(again, _bits(lk[:2]), _bits(lv[:2]), [3, 17])
    rk, rv = okv.load(again, [3, 17], 64)
    assert np.abs(rk - lk[:2]).max() <= np.abs(lk[:2]).max() / 8


def test_attention_closed_forms():
    d, n = 64, 9
    g = np.random.default_rng(1)
    v = g.standard_normal((n, 1, d))
    q0 = np.zeros((2, 2, d))
    out, lse, am = okv.attention(q0, np.zeros((n, 1, d)), v, 0.1)
    assert np.allclose(out[1, 0], v[:, 0].mean(axis=0)) and np.allclose(lse[1], np.log(n))
    assert np.allclose(out[0, 1], v[:-1, 0].mean(axis=0)) and np.allclose(lse[0], np.log(n - 1))
    out, lse, _ = okv.attention(q0, np.zeros((n, 1, d)), v, 0.1, window=2)
    assert np.allclose(out[0], v[6:8, 0].mean(axis=0))
    # more queries than keys: the first rows see nothing
    out, lse, _ = okv.attention(np.zeros((3, 1, d)), np.zeros((1, 1, d)), v[:1], 1.0)
    assert not out[:2].any() and np.isneginf(lse[:2]).all() and np.allclose(out[2, 0], v[0, 0])


@pytest.mark.parametrize("nq,n,hq,h", [(1, 7, 4, 2), (5, 40, 8, 2), (9, 9, 6, 6), (12, 30, 7, 1), (30, 12, 4, 4)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 4)])
def test_attention_against_a_library_softmax(nq, n, hq, h, causal, window):
    """Scale, logits, grouping of heads, masks and lse, by whole matrices in PyTorch's float64."""
    torch = pytest.importorskip("torch")
    d = 64
    g = np.random.default_rng(nq * n)
    q, k, v = g.standard_normal((nq, hq, d)), g.standard_normal((n, h, d)), g.standard_normal((n, h, d))
    held = g.random(n) < 0.8
    out, lse, mean = okv.attention(q, k, v, 0.3, causal, window, held)
    pos, tok = torch.arange(n - nq, n)[:, None], torch.arange(n)[None]
    mask = torch.from_numpy(held)[None].expand(nq, n).clone()
    if causal:
        mask &= tok <= pos
    if window:
        mask &= pos - tok < window
    tq, tk, tv = (torch.from_numpy(x).transpose(0, 1) for x in (q, k, v))
    tk, tv = (x.repeat_interleave(hq // h, dim=0) for x in (tk, tv))
    s = (tq @ tk.transpose(1, 2)).mul(0.3).masked_fill(~mask, float("-inf"))
    p = torch.softmax(s, dim=-1).nan_to_num(0.0)            # rows that see nothing: zeros
    assert np.allclose(out, (p @ tv).transpose(0, 1).numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(mean, (p @ tv.abs()).transpose(0, 1).numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(lse, torch.logsumexp(s, dim=-1).transpose(0, 1).numpy(), rtol=1e-12, atol=1e-12)
    seen = mask.any(dim=-1).numpy()
    assert np.isneginf(lse[~seen]).all() and not out[~seen].any() and np.isfinite(lse[seen]).all()
