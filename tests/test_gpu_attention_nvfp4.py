"""Attention over the NVFP4 cache against the float64 oracle on the values that the cache holds.

The tolerance of an output element: bf16 rounds it by at most 2^-8 of its value; the softmax
weights enter the second product rounded to f16, 2^-11 of each, so 2^-11 of the weighted mean of
|v|; float32 logits and sums are given 2^-12 of the same mean (a logit of size 32 is off by 2^-18,
sums over some thousand tokens by far less than 2^-13); weights below f16's smallest normal are
off by 2^-25 against a largest of at least 2^3, 2^-28 a token of the largest |v|.  lse: 2^-16 +
2^-20 of its value.
"""
import numpy as np
import pytest
import torch

from oracle import kvcache_nvfp4 as okv
from oracle.codecs import bf16_bits_to_f32, f32_to_bf16_bits_rne
from tests.helpers import DEV, bf16_bits_of, to_dev

pytestmark = pytest.mark.gpu

ql = pytest.importorskip("quantized_linear_layers_block_amd")
B = ql.binding


class Seqs:
    """Sequences with their cache: lens is a list of (query tokens, cached tokens)."""

    def __init__(self, lens, hq, h, d, page, seed, k_std=1.0, spare=2, poison=True):
        g = np.random.default_rng(seed)
        self.lens, self.hq, self.h, self.d, self.page = lens, hq, h, d, page
        counts = [max(1, -(-n // page)) for _, n in lens]
        pages = sum(counts) + spare
        perm = g.permutation(pages)
        self.table = np.full((len(lens), max(counts) + 1), 10 ** 6, np.int32)   # unused entries name no page
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = perm[at:at + c]
            at += c
        # unwritten memory holds the worst bytes: NaN scales, exponents of every kind
        fill = 0xFF if poison else 0
        self.data = okv.empty(pages, h, d, page, fill=fill)
        if poison:
            self.data[1::2] = 0xF6
        self.cache = ql.KVCacheNVFP4(torch.from_numpy(self.data.copy()).to(DEV), pages, h, d, page)
        for b, (_, n) in enumerate(lens):
            if n == 0:
                continue
            k = g.standard_normal((n, h, d)) * k_std * np.where(g.random((h, d)) < 0.05, 4, 0.7)
            v = g.standard_normal((n, h, d)) * np.exp2(g.integers(-3, 4, size=(n, h, 1)))
            s = torch.from_numpy(okv.sequence_slots(self.table[b], n, page)).to(DEV)
            ql.kv_store_nvfp4(to_dev(f32_to_bf16_bits_rne(k.astype(np.float32))),
                              to_dev(f32_to_bf16_bits_rne(v.astype(np.float32))), s, self.cache)
        torch.cuda.synchronize()
        self.data = self.cache.data.cpu().numpy()
        self.starts = np.concatenate([[0], np.cumsum([q for q, _ in lens])]).astype(np.int32)
        self.tq = int(self.starts[-1])
        self.q_bits = f32_to_bf16_bits_rne(g.standard_normal((max(self.tq, 1), hq, d)).astype(np.float32))
        self.q = to_dev(self.q_bits)[:self.tq]
        self.kv_lens = torch.tensor([n for _, n in lens], dtype=torch.int32, device=DEV)
        self.pt = torch.from_numpy(self.table).to(DEV)
        self.max_q = max(max(q for q, _ in lens), 1)
        self.uniform = len({q for q, _ in lens}) == 1

    def run(self, ragged=None, q=None, **kw):
        ragged = not self.uniform if ragged is None else ragged
        q = self.q if q is None else q
        lse = torch.full((q.shape[0], self.hq), 7.0, dtype=torch.float32, device=DEV)
        out = torch.full((q.shape[0], self.hq, self.d), 7.0, dtype=torch.bfloat16, device=DEV)
        starts = torch.from_numpy(self.starts).to(DEV) if ragged else None
        ql.attention_nvfp4(q, self.cache, self.pt, self.kv_lens, q_starts=starts, max_q_len=self.max_q, out=out, lse=lse,
                           **kw)
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, causal=True, window=0, scale=None, rows=24, seed=0, held=None, only=None, every=1):
        """Against the oracle, on at most `rows` query tokens of every `every`-th sequence (or on those
        of `only`)."""
        g = np.random.default_rng(seed)
        qf = bf16_bits_to_f32(self.q_bits).astype(np.float64)
        o, z = bf16_bits_to_f32(bf16_bits_of(out)).astype(np.float64), lse.cpu().numpy().astype(np.float64)
        scale = self.d ** -0.5 if scale is None else scale
        for b, (nq, n) in enumerate(self.lens):
            if nq == 0 or b % every:
                continue
            pick = np.arange(nq) if nq <= rows else np.unique(np.concatenate(
                [[0, 1, nq - 2, nq - 1], g.choice(nq, rows, replace=False)]))
            pick = pick if only is None else only
            k, v = (okv.load(self.data, okv.sequence_slots(self.table[b], n, self.page), self.d) if n
                    else (np.zeros((0, self.h, self.d)),) * 2)
            for i in pick:
                m = n - nq + i + 1 if causal else n      # the tokens up to this query's position
                m = max(m, 0)
                qq = qf[self.starts[b] + i][None]
                ro, rz, am = okv.attention(qq, k[:m], v[:m], scale, causal, window,
                                           None if held is None else held[b][:m])
                r = self.starts[b] + i
                vmax = np.abs(v[:m]).max() if m else 0.0
                tol = 2.0 ** -8 * np.abs(ro[0]) + (2.0 ** -11 + 2.0 ** -12) * am[0] + m * 2.0 ** -27 * vmax + 1e-30
                err = np.abs(o[r] - ro[0])
                assert (err <= tol).all(), f"sequence {b} query {i}: {err.max()} against {tol[err > tol].min()}"
                empty = np.isneginf(rz[0])
                assert (np.isneginf(z[r]) == empty).all()
                zr, zo = rz[0][~empty], z[r][~empty]
                assert (np.abs(zo - zr) <= 2.0 ** -16 + 2.0 ** -20 * np.abs(zr)).all()


@pytest.mark.parametrize("hq,h,d,page", [(28, 4, 128, 16), (8, 8, 64, 32), (16, 8, 256, 64), (64, 8, 128, 128),
                                         (5, 1, 128, 16), (32, 1, 64, 1024), (40, 2, 128, 16)])
def test_decode(hq, h, d, page):
    lens = [(1, n) for n in (1, 2, 15, 16, 17, 31, 32, 33, 100, 127, 128, 129, 300, 1023)]
    s = Seqs(lens, hq, h, d, page, hq + d)
    s.check(*s.run())


@pytest.mark.parametrize("nq,hq,h,d", [(2, 8, 2, 128), (5, 16, 8, 256), (8, 28, 4, 128), (3, 5, 5, 64)])
def test_a_few_query_tokens(nq, hq, h, d):
    s = Seqs([(nq, n) for n in (nq, nq + 1, 40, 64, 333)], hq, h, d, 16, nq)
    s.check(*s.run())
    s.check(*s.run(causal=False), causal=False)
    s.check(*s.run(window=7), window=7)


@pytest.mark.parametrize("lens,hq,h,d,page", [
    ([(129, 129)], 4, 2, 128, 16), ([(300, 300), (65, 1000)], 7, 1, 128, 64), ([(130, 700)], 8, 8, 64, 32),
    ([(70, 70), (300, 555)], 4, 2, 256, 16)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 100)])
def test_prompts(lens, hq, h, d, page, causal, window):
    s = Seqs(lens, hq, h, d, page, d + len(lens))
    s.check(*s.run(causal=causal, window=window), causal=causal, window=window)


@pytest.mark.parametrize("lens,hq,h,d,page", [
    ([(130, 3000)], 4, 2, 128, 64), ([(70, 2500), (200, 4000), (90, 90)], 3, 1, 128, 16), ([(300, 5000)], 2, 2, 64, 32),
    ([(66, 2100), (66, 40)], 2, 1, 256, 16)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1500)])
def test_prompt_pieces_far_into_long_contexts(lens, hq, h, d, page, causal, window):
    """Few units of many tokens, which are cut along the tokens and joined (a sequence with more
    queries than keys beside them: rows that see nothing in any part)."""
    s = Seqs(lens, hq, h, d, page, d + len(lens))
    s.check(*s.run(causal=causal, window=window), causal=causal, window=window, rows=10)


@pytest.mark.parametrize("batch,n,hq,h,d", [
    (20, 2000, 16, 8, 128),    # fewer units than workgroups: whole workgroups a unit
    (70, 1000, 16, 16, 64),    # more, over 64 sequences: shares that begin and end within units
    (70, 200, 16, 16, 64),     # the same with short shares
    (90, 900, 4, 2, 128),      # over 64 sequences in whole workgroups
    (33, 700, 4, 4, 256)])
def test_cuts_of_the_work(batch, n, hq, h, d):
    g = np.random.default_rng(batch + n)
    s = Seqs([(1, int(x)) for x in g.integers(n // 2, n + 1, batch)], hq, h, d, 64, n)
    every = 3 if batch > 64 else 1
    s.check(*s.run(), every=every)
    s.check(*s.run(window=n // 3), window=n // 3, every=every)


@pytest.mark.parametrize("window", [1 << 30, (1 << 31) - 1])
def test_largest_windows_with_more_queries_than_keys(window):
    for lens in ([(5, 3), (5, 40)], [(100, 60), (70, 0), (90, 200)]):
        s = Seqs(lens, 4, 2, 128, 16, 9)
        s.check(*s.run(window=window), window=window)


def test_bounds_that_pass_32_bits():
    """A table of 2^24 tokens a sequence for 300 sequences of 8 heads: the work could pass 2^31
    chunks, and the positions in it are kept in 64 bits."""
    lens = [(1, 900), (2, 77), (0, 5), (1, 3000)]
    s = Seqs(lens + [(0, 0)] * 295 + [(3, 300)], 16, 8, 128, 256, 1)
    wide = torch.full((len(s.lens), 1 << 16), -1, dtype=torch.int32, device=DEV)
    wide[:, :s.pt.shape[1]] = s.pt
    for s.pt, s.max_q in ((s.pt, 4), (wide, 4), (wide, 16384)):
        s.check(*s.run())


@pytest.mark.parametrize("nq,hq,h,d", [(12, 16, 2, 64), (16, 8, 1, 128), (9, 64, 8, 128), (65, 1, 1, 256)])
def test_around_a_hundred_rows_a_head(nq, hq, h, d):
    s = Seqs([(nq, n) for n in (nq, 40, 333, 1200)], hq, h, d, 32, nq)
    s.check(*s.run())
    s.check(*s.run(window=50), window=50)


@pytest.mark.parametrize("hq,h,d", [(1, 1, 64), (2, 2, 128)])
def test_prompts_of_many_sequences(hq, h, d):
    """Over 64 sequences, of all lengths: the units' order and the cuts along the tokens."""
    g = np.random.default_rng(d)
    lens = [(int(q), int(q + c)) for q, c in zip(g.integers(60, 300, 70), g.integers(0, 1500, 70))]
    s = Seqs(lens, hq, h, d, 64, d)
    s.check(*s.run(), rows=4)
    s.check(*s.run(window=400), window=400, rows=2)


def test_one_row_tile_and_decode_rows_agree():
    """The same queries as 64 rows and as 65 (the few-row kernel and the prompt kernel)."""
    for d in (64, 128, 256):
        s = Seqs([(65, 700)], 1, 1, d, 16, 40 + d)
        a, la = s.run()
        s.check(a, la)
        t = Seqs([(65, 700)], 1, 1, d, 16, 40 + d)
        t.starts = np.array([0, 64], np.int32)
        t.kv_lens -= 1
        t.max_q = 64
        b, lb = t.run(ragged=True)
        assert float((a[:64].float() - b[:64].float()).abs().max()) <= 2.0 ** -6 * float(a.float().abs().max())
        assert float((la[:64] - lb[:64]).abs().max()) <= 1e-4


@pytest.mark.parametrize("scale", [-0.05, 0.0, 3.0])
def test_prompt_scales_and_extreme_rows(scale):
    """Negative, zero and large scales; a zero, a tiny and an infinite query row; a NaN token."""
    s = Seqs([(100, 160)], 2, 1, 64, 16, 31)
    s.q_bits[3] = 0
    s.q_bits[5] = 0x0001                       # the smallest bf16
    s.q = to_dev(s.q_bits)
    out, lse = s.run(softmax_scale=scale)
    s.check(out, lse, scale=scale)
    s.q_bits[7, 1, 2] = 0x7F80
    s.q = to_dev(s.q_bits)
    k = f32_to_bf16_bits_rne(np.ones((1, 1, 64), np.float32))
    bad = k.copy()
    bad[0, 0, 9] = 0x7FC0
    slot = torch.from_numpy(okv.sequence_slots(s.table[0], 160, 16)[140:141]).to(DEV)
    ql.kv_store_nvfp4(to_dev(bad), to_dev(k), slot, s.cache)
    out2, lse2 = s.run(softmax_scale=scale)
    o, z = out2.float().cpu().numpy(), lse2.cpu().numpy()
    assert np.isnan(o[80:]).all() and np.isnan(z[80:]).all()            # query 80 is at position 140
    assert np.isnan(o[7, 1]).all() and np.isfinite(np.delete(o[:80], 7, axis=0)).all()
    # the token that changed is beside the others in its 16, which share factors: those rows against
    # the oracle again
    s.data = s.cache.data.cpu().numpy()
    s.check(out2, lse2, scale=scale, only=[0, 3, 5, 8, 20, 60, 70, 78, 79])


def test_mixed_batch_with_empty_sequences():
    lens = [(1, 500), (0, 40), (200, 260), (1, 1), (3, 0), (17, 17), (0, 0), (1, 0), (64, 640), (5, 2)]
    s = Seqs(lens, 8, 2, 128, 16, 5)
    s.check(*s.run())
    s.check(*s.run(window=33), window=33)


def test_rows_behind_the_last_sequence_are_left():
    s = Seqs([(3, 30), (1, 9), (70, 80)], 4, 2, 64, 16, 6)
    more = torch.cat([s.q, s.q[:5]])
    out, lse = s.run(ragged=True, q=more)
    s.check(out, lse)
    assert bool((out[s.tq:] == 7).all()) and bool((lse[s.tq:] == 7).all())


def test_long_context_and_spread_of_scales():
    """One long sequence beside short ones; strong logits, where few tokens carry the sum."""
    lens = [(1, 20000), (1, 3), (1, 1500)]
    s = Seqs(lens, 8, 4, 128, 64, 11, k_std=6.0)
    s.check(*s.run())
    s.check(*s.run(window=700), window=700)
    s.check(*s.run(softmax_scale=-0.02), scale=-0.02)


def test_values_of_very_different_size():
    """A weight near 1 on a tiny value row beside small weights on large ones, and the reverse:
    the value exponents join the softmax and must not lose either."""
    d, h, n = 64, 1, 48
    s = Seqs([(1, n)], 1, h, d, 16, 12, poison=False)
    g = np.random.default_rng(4)
    for ve, kv in [(-30, 8.0), (30, -8.0), (-90, 3.0), (60, -30.0)]:
        k = np.zeros((n, h, d))
        v = g.standard_normal((n, h, d))
        q = np.zeros((1, 1, d))
        q[0, 0, 0] = 8.0
        k[17, 0, 0] = kv
        v[17] *= 2.0 ** ve
        s.q_bits = f32_to_bf16_bits_rne(q.astype(np.float32))
        s.q = to_dev(s.q_bits)
        sl = torch.from_numpy(okv.sequence_slots(s.table[0], n, 16)).to(DEV)
        ql.kv_store_nvfp4(to_dev(f32_to_bf16_bits_rne(k.astype(np.float32))),
                          to_dev(f32_to_bf16_bits_rne(v.astype(np.float32))), sl, s.cache)
        out, lse = s.run(softmax_scale=1.0)
        s.data = s.cache.data.cpu().numpy()
        rk, rv = okv.load(s.data, okv.sequence_slots(s.table[0], n, 16), d)
        ro, rz, am = okv.attention(bf16_bits_to_f32(s.q_bits).astype(np.float64), rk, rv, 1.0)
        o = bf16_bits_to_f32(bf16_bits_of(out)).astype(np.float64)
        # A weight p is taken relative to the row's largest weight times value scale, w; what f16
        # cannot hold of it is at most 2^-25 where the largest is at least 2^3.  So a token is
        # off by at most 2^-28 of the largest-w token's share, times its own |vhat| <= 2688 in the
        # units 2^ev of that token's scale; 2688 2^ev is at most twice that row's largest value.
        top = np.argmax(np.log2(np.e) * rk[:, 0, 0] * 8.0 + np.log2(np.abs(rv[:, 0]).max(axis=1)))
        flush = n * 2.0 ** -28 * 2 * np.abs(rv[top]).max()
        ok = np.abs(o - ro) <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2.0 ** -12) * am + flush
        assert ok.all(), (ve, kv, o[~ok], ro[~ok])
        assert np.abs(lse.cpu().numpy() - rz).max() <= 2.0 ** -16 + 2.0 ** -20 * np.abs(rz).max()


def test_nan_tokens_reach_only_the_rows_that_see_them():
    lens = [(6, 40), (1, 33)]
    s = Seqs(lens, 4, 2, 64, 16, 13)
    k = np.ones((1, 2, 64), np.float32)
    v = np.ones((1, 2, 64), np.float32)
    v[0, 1, 3] = np.nan    # KV head 1, sequence 0, token 37: queries 3.. see it
    sl = torch.from_numpy(okv.sequence_slots(s.table[0], 38, 16)[37:]).to(DEV)
    ql.kv_store_nvfp4(to_dev(f32_to_bf16_bits_rne(k)), to_dev(np.where(np.isnan(v), 0x7FC0, f32_to_bf16_bits_rne(np.nan_to_num(v))).astype(np.uint16)),
                      sl, s.cache)
    s.q_bits[s.starts[1], 0, 0] = 0x7F80   # an infinite query
    s.q = to_dev(s.q_bits)[:s.tq]
    out, lse = s.run()
    o, z = out.float().cpu().numpy(), lse.cpu().numpy()
    assert np.isnan(o[3:6, 2:]).all() and np.isnan(z[3:6, 2:]).all()
    assert np.isfinite(o[:3]).all() and np.isfinite(o[:6, :2]).all() and np.isfinite(z[:3]).all()
    assert np.isnan(o[6, 0]).all() and np.isfinite(o[6, 1:]).all()


def test_bad_tables_are_cut_and_reported():
    s = Seqs([(1, 100), (1, 50), (1, 20)], 4, 2, 64, 16, 14)
    ws = torch.zeros(B.qlinear_attention_nvfp4_workspace(3, 3, 4, 2, 64, 1), dtype=torch.uint8, device=DEV)
    s.check(*s.run(ws=ws))
    assert ql.workspace_status(ws) == 0
    held = [np.ones(n, bool) for _, n in s.lens]
    good = s.table.copy()
    s.pt[0, 2], s.pt[1, 0] = -1, 10 ** 9
    held[0][32:48] = False
    held[1][:16] = False
    out, lse = s.run(ws=ws)
    assert ql.workspace_status(ws) == B.QLINEAR_STATUS_BAD_ITEM
    s.check(out, lse, held=held)
    # lengths beyond the table are cut to it, negative ones to nothing
    ws.zero_()
    s.pt = torch.from_numpy(good[:, :4].copy()).to(DEV)   # 64 tokens
    s.kv_lens = torch.tensor([2 ** 30, 50, -5], dtype=torch.int32, device=DEV)
    out, lse = s.run(ws=ws)
    assert ql.workspace_status(ws) == B.QLINEAR_STATUS_BAD_ITEM
    s.lens = [(1, 64), (1, 50), (1, 0)]
    s.check(out, lse)
    # query ranges outside q, or longer than max_q_len, are left out
    s = Seqs([(2, 30), (2, 30), (2, 30)], 4, 2, 64, 16, 15)
    ok = s.run()[0]
    s.starts = np.array([0, 2, 1, 9], np.int32)
    ws.zero_()
    out, _ = s.run(ragged=True, ws=torch.zeros(B.qlinear_attention_nvfp4_workspace(3, 6, 4, 2, 64, 2),
                                               dtype=torch.uint8, device=DEV))
    assert torch.equal(out[:2], ok[:2]) and bool((out[2:] == 7).all())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_q_starts_that_fall(d):
    """Sequences that overlap take more units than the call's sizes promise: reported, and nothing is
    touched outside out, lse and the workspace, whose last bytes a guard follows."""
    t, heads = 1000, 2
    s = Seqs([(t, t)] * 9, heads, heads, d, 64, d)
    q = s.q[:t].contiguous()
    starts = torch.tensor([0, t, 0, t, 0, t, 0, t, 0, t], dtype=torch.int32, device=DEV)
    need = B.qlinear_attention_nvfp4_workspace(9, t, heads, heads, d, t)
    ws = torch.zeros(need + 4096, dtype=torch.uint8, device=DEV)
    ws[need:] = 0x5A
    out = torch.full((t + 8, heads, d), 7.0, dtype=torch.bfloat16, device=DEV)
    B.qlinear_attention_nvfp4(s.cache.handle, q, s.pt, s.kv_lens, out[:t], ws[:need], starts, t, d ** -0.5)
    torch.cuda.synchronize()
    assert ql.workspace_status(ws) == B.QLINEAR_STATUS_BAD_ITEM
    assert (ws[need:] == 0x5A).all() and (out[t:] == 7.0).all()


@pytest.mark.parametrize("lens", [[(1, n) for n in (700, 3, 2500, 90)], [(100, 400), (1, 900)]])
def test_strides_workspace_reuse_and_reproducibility(lens):
    hq, h, d = 12, 4, 128
    s = Seqs(lens, hq, h, d, 32, 16)
    out, lse = s.run()
    s.check(out, lse)
    ws = torch.zeros(B.qlinear_attention_nvfp4_workspace(len(lens), s.tq, hq, h, d, s.max_q), dtype=torch.uint8,
                     device=DEV)
    fused = torch.zeros((s.tq, hq + 2 * h, d), dtype=torch.bfloat16, device=DEV)
    fused[:, :hq] = s.q
    wide = torch.full((s.tq, 2, hq, d), 3.0, dtype=torch.bfloat16, device=DEV)
    starts = torch.from_numpy(s.starts).to(DEV)
    for _ in range(3):
        lse2 = torch.empty_like(lse)
        ql.attention_nvfp4(fused[:, :hq], s.cache, s.pt, s.kv_lens, q_starts=starts, max_q_len=s.max_q, out=wide[:, 1],
                           lse=lse2, ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(wide[:, 1], out) and torch.equal(lse2, lse) and bool((wide[:, 0] == 3).all())
        assert ql.workspace_status(ws) == 0 and int(torch.count_nonzero(ws[256:B.QLINEAR_WS_RESERVED_BYTES])) == 0


def test_captured_decode_steps_replay():
    """A decode step as a user captures it: store the step's keys and values, attend.  Replays
    follow the lengths, slots and tensors as they are then, with eager work between."""
    hq, h, d, page = 8, 2, 128, 16
    s = Seqs([(1, n) for n in (900, 17, 64, 3000)], hq, h, d, page, 17)
    g = np.random.default_rng(3)
    k, v, q = (torch.empty((4, n, d), dtype=torch.bfloat16, device=DEV) for n in (h, h, hq))
    slots = torch.zeros(4, dtype=torch.int64, device=DEV)
    out = torch.empty_like(q)
    ws = torch.zeros(B.qlinear_attention_nvfp4_workspace(4, 4, hq, h, d, 1), dtype=torch.uint8, device=DEV)

    def step():
        ql.kv_store_nvfp4(k, v, slots, s.cache)
        ql.attention_nvfp4(q, s.cache, s.pt, s.kv_lens, out=out, ws=ws)

    def fresh(i):
        for t in (k, v, q):
            t.copy_(to_dev(f32_to_bf16_bits_rne(g.standard_normal(tuple(t.shape)).astype(np.float32))))
        lens = [900 + i % 12, 17 + i, 59 + i % 5, 2990 + i]
        s.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        slots.copy_(torch.tensor([okv.sequence_slots(s.table[b], n, page)[n - 1] for b, n in enumerate(lens)]))

    fresh(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(1, 5):
        fresh(i)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        eager = ql.attention_nvfp4(q, s.cache, s.pt, s.kv_lens)
        torch.cuda.synchronize()
        assert torch.equal(got, eager), f"replay {i}"
        s.lens = [(1, int(n)) for n in s.kv_lens.cpu()]
        s.data = s.cache.data.cpu().numpy()
        s.q_bits = bf16_bits_of(q)
        s.check(eager, ql_lse(s, q))


def ql_lse(s, q):
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=DEV)
    ql.attention_nvfp4(q, s.cache, s.pt, s.kv_lens, lse=lse)
    return lse


def test_other_stream():
    s = Seqs([(1, 400), (1, 30)], 4, 2, 64, 16, 18)
    want, _ = s.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ql.attention_nvfp4(s.q, s.cache, s.pt, s.kv_lens)
    side.synchronize()
    assert torch.equal(got, want)


def test_captured_mixed_batch_follows_starts_and_lengths():
    """Prompts and decode rows in one captured call: replays take the lengths and the query ranges
    that are on the device then, and give what an eager call gives, bit by bit."""
    lens = [(1, 900), (200, 1500), (70, 70), (1, 3), (40, 2000)]
    s = Seqs(lens, 8, 2, 128, 16, 23)
    starts = torch.from_numpy(s.starts).to(DEV)
    out, lse = torch.empty_like(s.q), torch.empty((s.tq, 8), dtype=torch.float32, device=DEV)
    ws = torch.zeros(B.qlinear_attention_nvfp4_workspace(5, s.tq, 8, 2, 128, 300), dtype=torch.uint8, device=DEV)

    def call(out, lse, ws=None):
        ql.attention_nvfp4(s.q, s.cache, s.pt, s.kv_lens, q_starts=starts, max_q_len=300, out=out, lse=lse, ws=ws)

    call(out, lse, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, lse, ws)
    for cut in ([1, 200, 70, 1, 40], [1, 1, 1, 1, 1], [60, 250, 1, 0, 1], [1, 200, 70, 1, 40]):
        q_lens = np.array(cut)
        starts.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)))
        s.lens = [(int(q), n) for q, (_, n) in zip(q_lens, lens)]
        s.starts = starts.cpu().numpy()
        out.fill_(float("nan"))
        lse.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        eager, eager_lse = torch.full_like(out, float("nan")), torch.full_like(lse, float("nan"))
        call(eager, eager_lse)
        torch.cuda.synchronize()
        used = int(s.starts[-1])
        assert torch.equal(out[:used], eager[:used]) and torch.equal(lse[:used], eager_lse[:used])
        assert torch.isnan(out[used:]).all() and torch.isnan(lse[used:]).all()
        s.check(out, lse, rows=8)


def test_two_calls_at_once():
    """On two streams, each with a workspace of its own."""
    a, b = Seqs([(1, 3000)] * 8, 16, 4, 128, 16, 31), Seqs([(150, 2500), (90, 800)], 8, 2, 64, 32, 32)
    want = [x.run()[0].clone() for x in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                starts = None if x.uniform else torch.from_numpy(x.starts).to(DEV)
                got[i].append(ql.attention_nvfp4(x.q, x.cache, x.pt, x.kv_lens, q_starts=starts, max_q_len=x.max_q))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_offsets_past_32_bits():
    """A cache of more than 4 GiB, with the sequence's pages at its end."""
    h, d, page = 8, 256, 1024
    per_page = h * page * (2 * (d // 2 + d // 16 + 1))
    pages = (5 << 30) // per_page
    cache = ql.KVCacheNVFP4.empty(pages, h, d, page, device=DEV)
    small = Seqs([(1, 1500)], 16, h, d, page, 19, spare=0, poison=False)
    cache.data[pages - 2:] = small.cache.data[:2]
    table = small.pt.clone()
    table[:, :2] += pages - 2
    want, _ = small.run()
    got = ql.attention_nvfp4(small.q, cache, table, small.kv_lens)
    slots = torch.from_numpy(okv.sequence_slots(small.table[0], 1500, page)).to(DEV)
    a, b = ql.kv_load_nvfp4(small.cache, slots)
    a2, b2 = ql.kv_load_nvfp4(cache, slots + (pages - 2) * page)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(a, a2) and torch.equal(b, b2)
    ql.kv_store_nvfp4(a, b, slots + (pages - 2) * page, cache)
    ql.kv_store_nvfp4(a, b, slots, small.cache)
    torch.cuda.synchronize()
    assert torch.equal(cache.data[pages - 2:], small.cache.data[:2])
