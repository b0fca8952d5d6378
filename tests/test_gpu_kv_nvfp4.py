"""The NVFP4 KV cache's store and load on the GPU: every byte of the cache against the oracle
(also the bytes that must not change), loaded values exact, bad slots and NaN tokens."""
import numpy as np
import pytest
import torch

from oracle import kvcache_nvfp4 as okv
from oracle.codecs import bf16_bits_to_f32, f32_to_bf16_bits_rne
from tests.helpers import DEV, bf16_bits_of, to_dev

pytestmark = pytest.mark.gpu

ql = pytest.importorskip("quantized_linear_layers_block_amd")
B = ql.binding


def _rows(seed, t, h, d):
    g = np.random.default_rng(seed)
    x = g.standard_t(3, size=(t, h, d))
    x *= np.exp2(g.integers(-6, 6, size=(t, h, 1)))
    x[0, 0] = 0.0
    x[-1, -1, 1:] = -0.0
    if t > 3:
        x[1, -1] *= 1e-35
        x[2, 0] *= 1e30
        x[3, 0] = np.exp2(g.integers(-140, 127, size=d))                     # block scales from 0 to 448
        x[3, -1] = g.integers(-28, 29, size=d) * 0.25 * (2688.0 / 7) / 384   # ties of the element grid
    return f32_to_bf16_bits_rne(x.astype(np.float32))


def _loaded(k):
    return bf16_bits_to_f32(bf16_bits_of(k)).astype(np.float64)


@pytest.mark.parametrize("t,h,d,page,pages", [(1, 1, 128, 16, 1), (5, 2, 64, 16, 3), (37, 8, 128, 64, 3),
                                              (33, 3, 256, 32, 2), (200, 5, 128, 16, 20), (9, 1, 64, 1024, 1),
                                              (130, 4, 256, 128, 2)])
@pytest.mark.parametrize("run", [False, True])
def test_store_load_bytes(t, h, d, page, pages, run):
    """run: consecutive slots from an odd one, as a prompt's; else scattered ones."""
    k, v = _rows(t + d, t, h, d), _rows(t + d + 1, t, h, d)
    g = np.random.default_rng(d)
    if run:
        slots = np.arange(t) + (3 if pages * page >= t + 3 else 0)
    else:
        slots = g.permutation(pages * page)[:t]
    ref = okv.empty(pages, h, d, page, fill=0xAB)
    cache = ql.KVCacheNVFP4(torch.from_numpy(ref.copy()).to(DEV), pages, h, d, page)
    sl = torch.from_numpy(slots.astype(np.int64)).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ql.kv_store_nvfp4(to_dev(k), to_dev(v), sl, cache, status)
    back = sl.flip(0).contiguous()
    lk, lv = ql.kv_load_nvfp4(cache, back, status_word=status)
    torch.cuda.synchronize()
    okv.store(ref, k, v, slots)
    got = cache.data.cpu().numpy()
    assert np.array_equal(got, ref), np.argwhere(got != ref)[:5]
    rk, rv = okv.load(ref, slots[::-1], d)
    assert np.array_equal(_loaded(lk), rk) and np.array_equal(_loaded(lv), rv)
    assert status.item() == 0


def test_parts_of_a_fused_projection_and_single_outputs():
    t, h, d = 21, 2, 128
    qkv = to_dev(_rows(3, t, 8 + 2 * h, d))
    k, v = qkv[:, 8:8 + h], qkv[:, 8 + h:]
    slots = torch.from_numpy(np.random.default_rng(2).permutation(64)[:t].astype(np.int64)).to(DEV)
    a, b = (ql.KVCacheNVFP4(torch.zeros((4, h, 1, 18 * d + 32), dtype=torch.uint8, device=DEV), 4, h, d, 16)
            for _ in range(2))
    ql.kv_store_nvfp4(k, v, slots, a)
    ql.kv_store_nvfp4(k.contiguous(), v.contiguous(), slots, b)
    assert torch.equal(a.data, b.data)
    wide = torch.full((t, 3, h, d), 7.0, dtype=torch.bfloat16, device=DEV)
    ql.kv_load_nvfp4(a, slots, k_out=wide[:, 0], v_out=wide[:, 2])
    lk, lv = ql.kv_load_nvfp4(a, slots)
    assert torch.equal(wide[:, 0], lk) and torch.equal(wide[:, 2], lv) and bool((wide[:, 1] == 7).all())
    only = torch.empty_like(lk)
    B.qlinear_kv_load_nvfp4(a.handle, slots, k_out=only)
    assert torch.equal(only, lk)
    B.qlinear_kv_load_nvfp4(a.handle, slots, v_out=only)
    assert torch.equal(only, lv)


def test_slots_outside_and_nan_tokens():
    t, h, d = 5, 3, 64
    k, v = _rows(8, t, h, d), _rows(9, t, h, d)
    k[1, 1, 63], v[2, 0, 0], v[3, 2, 5] = 0x7F80, 0x7FC0, 0xFF80
    slots = np.array([5, 0, 31, 17, 32])
    ref = okv.empty(2, h, d, 16, fill=0x55)
    cache = ql.KVCacheNVFP4(torch.from_numpy(ref.copy()).to(DEV), 2, h, d, 16)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    sl = torch.from_numpy(slots).to(DEV)
    ql.kv_store_nvfp4(to_dev(k), to_dev(v), sl, cache, status)
    torch.cuda.synchronize()
    assert status.item() == B.QLINEAR_STATUS_BAD_ITEM | B.QLINEAR_STATUS_NONFINITE
    okv.store(ref, k, v, slots)
    assert np.array_equal(cache.data.cpu().numpy(), ref)
    status.zero_()
    sl2 = torch.tensor([31, -1, 0, 2 ** 40, 17], dtype=torch.int64, device=DEV)
    lk, lv = ql.kv_load_nvfp4(cache, sl2, status_word=status)
    torch.cuda.synchronize()
    assert status.item() == B.QLINEAR_STATUS_BAD_ITEM
    rk, rv = okv.load(ref, sl2.cpu().numpy(), d)
    assert np.array_equal(_loaded(lk), rk, equal_nan=True) and np.array_equal(_loaded(lv), rv, equal_nan=True)
    assert np.isnan(rk[0, 0]).all() and not rk[1].any()


def test_no_tokens():
    cache = ql.KVCacheNVFP4.empty(2, 2, 64, 16, device=DEV)
    cache.data.fill_(1)
    x = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    s = torch.empty(0, dtype=torch.int64, device=DEV)
    ql.kv_store_nvfp4(x, x, s, cache)
    k, v = ql.kv_load_nvfp4(cache, s)
    assert k.shape == (0, 2, 64) and v.shape == (0, 2, 64) and bool((cache.data == 1).all())
