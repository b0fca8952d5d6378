"""Attention over the NVFP4 cache where keys and values lie far apart in size, against the float64
oracle on the values that the cache holds; the bounds are those of test_gpu_attention_nvfp4.py.

Both kernels (few query rows a sequence, and prompts), whole and cut into parts that are joined.
The sum of the weights, and so lse, must not depend on the values at all.
"""
import numpy as np
import pytest
import torch

from oracle import kvcache_nvfp4 as okv
from oracle.codecs import f32_to_bf16_bits_rne
from tests.helpers import DEV, to_dev
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
