"""What the NVFP4 KV cache's entry points refuse, on the host: the C ABI's argument errors
(nothing is launched) and the package helpers' checks that need no GPU."""
import ctypes

import pytest

b = pytest.importorskip("quantized_linear_layers_block_amd").binding
L = b.LIB
FAKE = 0x10000  # an aligned, never-dereferenced address


def _cache(data=FAKE, pages=4, page_size=64, heads=8, head_dim=128):
    return b.KvNvfp4(data, pages, page_size, heads, head_dim, 0)


def test_cache_sizes():
    assert b.qlinear_kv_nvfp4_bytes(4, 64, 8, 128) == 4 * 64 * 8 * 146
    assert b.qlinear_kv_nvfp4_bytes(1, 16, 1, 64) == 18 * 64 + 32
    for bad in [(0, 64, 8, 128), (4, 8, 8, 128), (4, 48, 8, 128), (4, 2048, 8, 128), (4, 64, 0, 128), (4, 64, 8, 96),
                (4, 64, 8, 512), (1 << 40, 64, 8, 128), (4, 64, 65536, 128)]:
        assert b.qlinear_kv_nvfp4_bytes(*bad) == 0, bad


def test_store_load_errors():
    def st(cache=_cache(), k=FAKE, ks=1024, v=FAKE, vs=1024, t=4, slots=FAKE, status=None):
        return L.qlinear_kv_store_nvfp4(ctypes.byref(cache), k, ks, v, vs, t, slots, status, None)

    assert L.qlinear_kv_store_nvfp4(None, FAKE, 1024, FAKE, 1024, 4, FAKE, None, None) == b.QL_ERR_NULL
    assert st(_cache(data=None)) == b.QL_ERR_NULL
    assert st(k=None) == b.QL_ERR_NULL and st(v=None) == b.QL_ERR_NULL and st(slots=None) == b.QL_ERR_NULL
    assert st(_cache(head_dim=96)) == b.QL_ERR_SHAPE and st(_cache(page_size=24)) == b.QL_ERR_SHAPE
    assert st(_cache(pages=0)) == b.QL_ERR_SHAPE and st(_cache(heads=0)) == b.QL_ERR_SHAPE
    assert st(ks=1016) == b.QL_ERR_SHAPE and st(vs=1028) == b.QL_ERR_SHAPE and st(t=-1) == b.QL_ERR_SHAPE
    assert st(t=1 << 31, ks=1 << 20) == b.QL_ERR_SHAPE
    assert st(_cache(data=FAKE + 8)) == b.QL_ERR_ALIGN and st(k=FAKE + 2) == b.QL_ERR_ALIGN
    assert st(slots=FAKE + 4) == b.QL_ERR_ALIGN and st(status=FAKE + 2) == b.QL_ERR_ALIGN
    assert st(t=0) == b.QL_OK

    def ld(cache=_cache(), slots=FAKE, t=4, k=FAKE, ks=1024, v=FAKE, vs=1024, status=None):
        return L.qlinear_kv_load_nvfp4(ctypes.byref(cache), slots, t, k, ks, v, vs, status, None)

    assert ld(slots=None) == b.QL_ERR_NULL and ld(k=None, v=None) == b.QL_ERR_NULL
    assert ld(t=-1) == b.QL_ERR_SHAPE and ld(ks=8) == b.QL_ERR_SHAPE and ld(k=None, vs=8) == b.QL_ERR_SHAPE
    assert ld(v=FAKE + 4) == b.QL_ERR_ALIGN
    assert ld(t=0, k=None) == b.QL_OK


def test_attention_errors():
    need = b.qlinear_attention_nvfp4_workspace(2, 2, 32, 8, 128, 1)
    assert need >= b.QLINEAR_WS_RESERVED_BYTES

    def at(cache=_cache(), batch=2, mq=1, tq=2, starts=None, lens=FAKE, table=FAKE, ts=5, tp=5, q=FAKE, qs=4096, hq=32,
           scale=0.1, causal=1, window=0, out=FAKE, os=4096, lse=None, ws=FAKE, wsb=1 << 40):
        seqs = b.AttnBatch(batch, mq, tq, starts, lens, table, ts, tp)
        return L.qlinear_attention_nvfp4(ctypes.byref(cache), ctypes.byref(seqs), q, qs, hq, scale, causal, window, out,
                                         os, lse, ws, wsb, None)

    assert at(q=None) == b.QL_ERR_NULL and at(out=None) == b.QL_ERR_NULL
    assert at(lens=None) == b.QL_ERR_NULL and at(table=None) == b.QL_ERR_NULL
    assert at(_cache(data=None)) == b.QL_ERR_NULL
    assert at(_cache(head_dim=80)) == b.QL_ERR_SHAPE
    assert at(batch=0, tq=0) == b.QL_ERR_SHAPE and at(batch=65536, tq=65536) == b.QL_ERR_SHAPE
    assert at(mq=0, tq=0) == b.QL_ERR_SHAPE and at(tq=3) == b.QL_ERR_SHAPE
    assert at(hq=30) == b.QL_ERR_SHAPE and at(hq=0) == b.QL_ERR_SHAPE
    assert at(mq=1 << 25, starts=FAKE) == b.QL_ERR_SHAPE
    assert at(tp=0) == b.QL_ERR_SHAPE and at(ts=1 << 24, tp=1 << 24) == b.QL_ERR_SHAPE
    assert at(ts=4) == b.QL_ERR_SHAPE and at(ts=0) == b.QL_ERR_SHAPE   # rows that overlap
    assert at(ts=1 << 60) == b.QL_ERR_SHAPE
    assert at(_cache(heads=512), batch=16384, mq=65, tq=16384 * 65, hq=512, qs=65536, os=65536) == b.QL_ERR_SHAPE   # launch
    assert at(qs=4088) == b.QL_ERR_SHAPE and at(os=4100) == b.QL_ERR_SHAPE
    assert at(window=-1) == b.QL_ERR_ARG and at(window=5, causal=0) == b.QL_ERR_ARG
    assert at(scale=float("inf")) == b.QL_ERR_ARG and at(scale=float("nan")) == b.QL_ERR_ARG
    assert at(scale=3e38) == b.QL_ERR_ARG   # finite, but not times log2(e)
    assert at(q=FAKE + 8) == b.QL_ERR_ALIGN and at(out=FAKE + 2) == b.QL_ERR_ALIGN and at(lse=FAKE + 2) == b.QL_ERR_ALIGN
    assert at(starts=FAKE + 2) == b.QL_ERR_ALIGN and at(table=FAKE + 1) == b.QL_ERR_ALIGN
    assert at(ws=None) == b.QL_ERR_WORKSPACE and at(wsb=need - 1) == b.QL_ERR_WORKSPACE
    assert at(ws=FAKE + 8) == b.QL_ERR_ALIGN
    for bad in [(0, 2, 32, 8, 128, 1), (2, 0, 32, 8, 128, 1), (2, 2, 31, 8, 128, 1), (2, 2, 32, 8, 96, 1),
                (2, 2, 32, 8, 128, 0)]:
        assert b.qlinear_attention_nvfp4_workspace(*bad) == 0, bad


def test_helpers_refuse_host_tensors_and_wrong_sizes():
    torch = pytest.importorskip("torch")
    import quantized_linear_layers_block_amd as ql
    with pytest.raises(ValueError):
        ql.KVCacheNVFP4.empty(2, 2, 96, device="cpu")
    with pytest.raises(ValueError):
        ql.KVCacheNVFP4.empty(2, 2, 64, page_size=24, device="cpu")
    with pytest.raises(ValueError):
        ql.KVCacheNVFP4(torch.zeros(100, dtype=torch.uint8), 2, 2, 64, 16)
    c = ql.KVCacheNVFP4.empty(2, 2, 64, page_size=16, device="cpu")
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        ql.kv_store_nvfp4(x, x, slots, c)
    with pytest.raises(ValueError):
        ql.kv_load_nvfp4(c, slots)
    with pytest.raises(ValueError):
        ql.attention_nvfp4(x, c, torch.zeros((3, 1), dtype=torch.int32), torch.ones(3, dtype=torch.int32))


def test_package_imports_with_a_pytorch_for_hosts_alone():
    """The size queries and refusals need no GPU, nor the PyTorch internals of a GPU build."""
    import os
    import subprocess
    import sys
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getDevice'): del torch._C._cuda_getDevice\n"
            "import quantized_linear_layers_block_amd as ql\n"
            "assert ql.KVCacheNVFP4.empty(2, 2, 64, 16, device='cpu').data.numel() == 2 * 2 * (18 * 64 + 32)\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
