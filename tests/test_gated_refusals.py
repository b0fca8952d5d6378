"""What the gated block's entry points refuse, on the host: the C ABI's argument errors (nothing is
launched) and the package helpers' checks that need no GPU."""
import ctypes

import pytest

b = pytest.importorskip("quantized_linear_layers_block_amd").binding
L = b.LIB
FAKE = 0x10000  # an aligned, never-dereferenced address


def _w(fmt=b.QL_FP8_BLOCK128, n=256, k=512, codes=FAKE, scales=FAKE):
    return b.QWeight(fmt, 0, n, k, codes, scales, None)


def test_gated_forward_errors():
    need = b.qlinear_gated_forward_workspace(4, 256, 512)
    assert need >= b.QLINEAR_WS_RESERVED_BYTES + 4 * 256 * 4
    assert b.qlinear_gated_forward_workspace(300, 256, 512) >= b.QLINEAR_WS_RESERVED_BYTES
    for bad in [(0, 256, 512), (4, 200, 512), (4, 256, 500), (4, 0, 512), (4, 256, 0), (4, 128, 1 << 24),
                ((1 << 24) + 1, 256, 512), (1, 1 << 23, 128), (64, 1 << 23, 128)]:
        assert b.qlinear_gated_forward_workspace(*bad) == 0, bad

    def f(gate=_w(), up=_w(), xq=FAKE, sx=FAKE, m=4, h=FAKE, hq=None, sh=None, gu=None, ws=FAKE, wsb=1 << 40):
        return L.qlinear_gated_forward(ctypes.byref(gate), ctypes.byref(up), xq, sx, m, h, hq, sh, gu, ws, wsb, None)

    assert L.qlinear_gated_forward(None, ctypes.byref(_w()), FAKE, FAKE, 4, FAKE, None, None, None, FAKE, 1 << 40,
                                   None) == b.QL_ERR_NULL
    assert L.qlinear_gated_forward(ctypes.byref(_w()), None, FAKE, FAKE, 4, FAKE, None, None, None, FAKE, 1 << 40,
                                   None) == b.QL_ERR_NULL
    assert f(_w(codes=None)) == b.QL_ERR_NULL and f(up=_w(scales=None)) == b.QL_ERR_NULL
    assert f(xq=None) == b.QL_ERR_NULL and f(sx=None) == b.QL_ERR_NULL and f(h=None) == b.QL_ERR_NULL
    assert f(hq=FAKE) == b.QL_ERR_NULL
    nv = b.QWeight(b.QL_NVFP4, 0, 256, 512, FAKE, FAKE, FAKE)
    assert f(nv, nv) == b.QL_ERR_FORMAT and f(up=_w(b.QL_FP8_POW2)) == b.QL_ERR_FORMAT and f(_w(9)) == b.QL_ERR_FORMAT
    assert f(up=_w(n=384)) == b.QL_ERR_SHAPE and f(up=_w(k=384)) == b.QL_ERR_SHAPE
    assert f(_w(n=200), _w(n=200)) == b.QL_ERR_SHAPE and f(m=0) == b.QL_ERR_SHAPE and f(m=-5) == b.QL_ERR_SHAPE
    assert f(m=(1 << 24) + 1) == b.QL_ERR_SHAPE
    assert f(_w(n=128, k=1 << 24), _w(n=128, k=1 << 24)) == b.QL_ERR_SHAPE
    assert f(_w(codes=FAKE + 8)) == b.QL_ERR_ALIGN and f(up=_w(scales=FAKE + 4)) == b.QL_ERR_ALIGN
    for name in ("xq", "sx", "h", "gu", "ws"):
        assert f(**{name: FAKE + 8}) == b.QL_ERR_ALIGN, name
    assert f(hq=FAKE + 4, sh=FAKE) == b.QL_ERR_ALIGN and f(hq=FAKE, sh=FAKE + 4) == b.QL_ERR_ALIGN
    assert f(ws=None) == b.QL_ERR_WORKSPACE and f(wsb=need - 1) == b.QL_ERR_WORKSPACE


def test_gated_backward_errors():
    need = b.qlinear_gated_backward_workspace(5, 256, 512)
    assert need >= 2 * 5 * 512 * 2
    for bad in [(0, 256, 512), (5, 100, 512), (5, 256, 64), (5, 1 << 22, 128), (5, 128, 1 << 22)]:
        assert b.qlinear_gated_backward_workspace(*bad) == 0, bad

    def f(gate=_w(), up=_w(), dh=FAKE, gu=FAKE, x=FAKE, m=5, dx=FAKE, dg=FAKE, du=FAKE, ws=FAKE, wsb=1 << 40):
        return L.qlinear_gated_backward(ctypes.byref(gate), ctypes.byref(up), dh, gu, x, m, dx, dg, du, ws, wsb, None)

    assert f(dh=None) == b.QL_ERR_NULL and f(gu=None) == b.QL_ERR_NULL and f(x=None) == b.QL_ERR_NULL
    assert f(dx=None, dg=None, du=None) == b.QL_ERR_NULL and f(dg=None) == b.QL_ERR_NULL and f(du=None) == b.QL_ERR_NULL
    assert f(_w(codes=None)) == b.QL_ERR_NULL
    nv = b.QWeight(b.QL_NVFP4, 0, 256, 512, FAKE, FAKE, FAKE)
    assert f(nv, nv) == b.QL_ERR_FORMAT and f(up=_w(b.QL_FP8_POW2)) == b.QL_ERR_FORMAT
    assert f(up=_w(n=128)) == b.QL_ERR_SHAPE and f(m=0) == b.QL_ERR_SHAPE and f(m=(1 << 24) + 1) == b.QL_ERR_SHAPE
    assert f(_w(n=128, k=1 << 22), _w(n=128, k=1 << 22)) == b.QL_ERR_SHAPE
    for name in ("dh", "gu", "x", "dx", "dg", "du", "ws"):
        assert f(**{name: FAKE + 8}) == b.QL_ERR_ALIGN, name
    assert f(ws=None) == b.QL_ERR_WORKSPACE and f(wsb=need - 1) == b.QL_ERR_WORKSPACE


def test_helpers_refuse():
    torch = pytest.importorskip("torch")
    import quantized_linear_layers_block_amd as ql
    w = ql.FP8Weight.empty(128, 256, device="cpu")
    xq, sx = torch.zeros((3, 256), dtype=torch.uint8), torch.zeros((3, 2))
    with pytest.raises(ValueError):   # not on the GPU
        ql.gated_forward(w, w, xq, sx)
    with pytest.raises(TypeError):
        ql.gated_forward(ql.NVFP4Weight.empty(128, 256, device="cpu"), w, xq, sx)
    with pytest.raises(ValueError):
        ql.gated_forward_fp8(w, ql.FP8Weight.empty(256, 256, device="cpu"), xq, sx)
    with pytest.raises(ValueError):
        ql.gated_forward(w, ql.FP8Weight.empty(128, 256, device="cpu", pow2=True), xq, sx)
    dh = torch.zeros((3, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ql.gated_backward(w, w, dh, dh)


def test_launch_limits():
    """More than 2^32 - 1 threads cannot be launched: refused, not left to the launch to fail."""
    assert b.qlinear_gated_forward_workspace(1 << 24, 4096, 128) > 0
    assert b.qlinear_gated_forward_workspace(1 << 24, 1 << 15, 128) == 0
    assert b.qlinear_gated_backward_workspace((1 << 24) - 64, 128, 4096) > 0
    assert b.qlinear_gated_backward_workspace((1 << 24) - 32, 128, 4096) == 0
    assert b.qlinear_gated_backward_workspace(1 << 24, 128, 128) == 0
    w = _w(n=128, k=128)
    assert L.qlinear_gated_backward(ctypes.byref(w), ctypes.byref(w), FAKE, FAKE, FAKE, 1 << 24, FAKE, FAKE, FAKE, FAKE,
                                    1 << 60, None) == b.QL_ERR_SHAPE
