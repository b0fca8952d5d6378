"""Calls of the NVFP4 attention helper at the edge of what its arguments allow."""
import pytest
import torch

from tests.helpers import DEV
from tests.test_gpu_attention_nvfp4 import Seqs

pytestmark = pytest.mark.gpu

ql = pytest.importorskip("quantized_linear_layers_block_amd")


@pytest.mark.parametrize("batch,starts", [(0, False), (0, True), (3, True), (3, False)])
def test_no_query_tokens(batch, starts):
    """As store and load of no tokens: nothing is launched, an empty result."""
    cache = ql.KVCacheNVFP4.empty(2, 2, 64, 16, device=DEV)
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    table = torch.zeros((batch, 1), dtype=torch.int32, device=DEV)
    lens = torch.ones(batch, dtype=torch.int32, device=DEV)
    kw = dict(q_starts=torch.zeros(batch + 1, dtype=torch.int32, device=DEV), max_q_len=4) if starts else {}
    lse = torch.empty((0, 4), dtype=torch.float32, device=DEV)
    out = ql.attention_nvfp4(q, cache, table, lens, lse=lse, **kw)
    assert out.shape == (0, 4, 64) and out.dtype == torch.bfloat16
    given = torch.empty_like(q)
    assert ql.attention_nvfp4(q, cache, table, lens, out=given, **kw) is given
    # the arguments are still looked at
    with pytest.raises(TypeError):
        ql.attention_nvfp4(q, cache, table, lens.to(torch.int64), **kw)
    with pytest.raises(ValueError):
        ql.attention_nvfp4(torch.empty((0, 3, 64), dtype=torch.bfloat16, device=DEV), cache, table, lens, **kw)


def test_queries_of_no_sequence_are_refused():
    cache = ql.KVCacheNVFP4.empty(2, 2, 64, 16, device=DEV)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ql.QlinearError):
        ql.attention_nvfp4(q, cache, torch.zeros((0, 1), dtype=torch.int32, device=DEV),
                           torch.zeros(0, dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("lens,hq,h,d", [([(1, 3000), (1, 70)], 8, 2, 128), ([(4, 900)] * 3, 16, 4, 64),
                                         ([(1, 9000)], 4, 1, 64),             # joined by the second kernel
                                         ([(200, 2500), (3, 40), (90, 90)], 4, 2, 128), ([(150, 400)], 2, 2, 256)])
def test_the_output_in_place_of_the_queries(lens, hq, h, d):
    s = Seqs(lens, hq, h, d, 32, 5)
    want, lse = s.run()
    q = s.q.clone()
    starts = None if s.uniform else torch.from_numpy(s.starts).to(DEV)
    lse2 = torch.empty_like(lse)
    ql.attention_nvfp4(q, s.cache, s.pt, s.kv_lens, q_starts=starts, max_q_len=s.max_q, out=q, lse=lse2)
    torch.cuda.synchronize()
    assert torch.equal(q, want) and torch.equal(lse2, lse)


def test_sequences_that_share_pages():
    """A common prefix held once, a page twice in one sequence, and two sequences alike."""
    s = Seqs([(1, 200), (1, 200), (70, 200)], 4, 2, 64, 32, 6)
    s.table[1] = s.table[0]
    s.table[2, :3] = s.table[0, :3]
    s.table[2, 4] = s.table[2, 3]
    s.pt = torch.from_numpy(s.table).to(DEV)
    s.check(*s.run())


def test_numbers_that_pass_32_bits_are_refused():
    s = Seqs([(1, 20)], 2, 1, 64, 16, 7)
    for kw in (dict(window=1 << 31), dict(window=4 - (1 << 32)), dict(max_q_len=(1 << 32) + 1), dict(max_q_len=1 - (1 << 32))):
        with pytest.raises((ValueError, ql.QlinearError)):
            ql.attention_nvfp4(s.q, s.cache, s.pt, s.kv_lens, **kw)
