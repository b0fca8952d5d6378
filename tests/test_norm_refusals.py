"""What the norm's entry points refuse, on the host: the C ABI's argument errors (nothing is
launched) and the package helpers' checks that need no GPU."""
import pytest

b = pytest.importorskip("quantized_linear_layers_block_amd").binding
L = b.LIB
FAKE = 0x10000  # an aligned, never-dereferenced address


def test_norm_errors():
    def f(x=FAKE, xs=256, r=None, rs=256, w=FAKE, eps=1e-6, m=4, k=256, h=None, hs=256, y=FAKE, fmt=0, yq=None, sy=None):
        return L.qlinear_rms_norm(x, xs, r, rs, w, eps, m, k, h, hs, y, fmt, yq, sy, None)

    assert f(x=None) == b.QL_ERR_NULL and f(w=None) == b.QL_ERR_NULL and f(y=None) == b.QL_ERR_NULL
    assert f(r=FAKE) == b.QL_ERR_NULL   # a residual needs a place for the sum
    assert f(fmt=b.QL_FP8_BLOCK128, yq=FAKE) == b.QL_ERR_NULL
    assert f(fmt=b.QL_NVFP4, yq=FAKE, sy=FAKE) == b.QL_ERR_FORMAT and f(yq=FAKE, sy=FAKE) == b.QL_ERR_FORMAT
    assert f(m=0) == b.QL_ERR_SHAPE and f(m=-1) == b.QL_ERR_SHAPE and f(m=(1 << 24) + 1) == b.QL_ERR_SHAPE
    assert f(k=0) == b.QL_ERR_SHAPE and f(k=252, xs=256) == b.QL_ERR_SHAPE
    assert f(k=65536 + 8, xs=1 << 20) == b.QL_ERR_SHAPE
    assert f(k=264, xs=264, fmt=b.QL_FP8_POW2, yq=FAKE, sy=FAKE) == b.QL_ERR_SHAPE
    assert f(xs=248) == b.QL_ERR_SHAPE and f(xs=260) == b.QL_ERR_SHAPE and f(xs=1 << 60) == b.QL_ERR_SHAPE
    assert f(r=FAKE, rs=0, h=FAKE) == b.QL_ERR_SHAPE and f(h=FAKE, hs=0) == b.QL_ERR_SHAPE
    for eps in (0.0, -1e-6, float("inf"), float("nan")):
        assert f(eps=eps) == b.QL_ERR_ARG
    assert f(x=FAKE + 8) == b.QL_ERR_ALIGN and f(w=FAKE + 2) == b.QL_ERR_ALIGN and f(y=FAKE + 4) == b.QL_ERR_ALIGN
    assert f(r=FAKE + 8, h=FAKE) == b.QL_ERR_ALIGN and f(h=FAKE + 8) == b.QL_ERR_ALIGN
    assert f(fmt=b.QL_FP8_POW2, yq=FAKE + 8, sy=FAKE) == b.QL_ERR_ALIGN
    assert f(fmt=b.QL_FP8_POW2, yq=FAKE, sy=FAKE + 1) == b.QL_ERR_ALIGN


def test_norm_backward_errors():
    need = b.qlinear_rms_norm_backward_workspace(4, 256)
    assert need >= 4 * 256 * 4
    for bad in [(0, 256), (4, 0), (4, 100), (4, 65544), ((1 << 24) + 1, 256)]:
        assert b.qlinear_rms_norm_backward_workspace(*bad) == 0

    def f(dy=FAKE, dys=256, h=FAKE, hs=256, w=FAKE, eps=1e-6, dh=None, dhs=256, m=4, k=256, dx=FAKE, dxs=256, dw=FAKE,
          ws=FAKE, wsb=1 << 30):
        return L.qlinear_rms_norm_backward(dy, dys, h, hs, w, eps, dh, dhs, m, k, dx, dxs, dw, ws, wsb, None)

    for name in ("dy", "h", "w", "dx"):
        assert f(**{name: None}) == b.QL_ERR_NULL, name
    assert f(m=0) == b.QL_ERR_SHAPE and f(k=12) == b.QL_ERR_SHAPE
    for name in ("dys", "hs", "dxs"):
        assert f(**{name: 8}) == b.QL_ERR_SHAPE, name
    assert f(dh=FAKE, dhs=8) == b.QL_ERR_SHAPE
    assert f(eps=0.0) == b.QL_ERR_ARG
    for name in ("dy", "h", "w", "dx", "dh", "dw", "ws"):
        assert f(**{name: FAKE + 8}) == b.QL_ERR_ALIGN, name
    assert f(ws=None) == b.QL_ERR_WORKSPACE and f(wsb=need - 1) == b.QL_ERR_WORKSPACE


def test_helpers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    import quantized_linear_layers_block_amd as ql
    x, w = torch.zeros((3, 128), dtype=torch.bfloat16), torch.ones(128, dtype=torch.bfloat16)
    for call in (lambda: ql.rms_norm(x, w), lambda: ql.rms_norm_fp8(x, w), lambda: ql.rms_norm_backward(x, x, w)):
        with pytest.raises(ValueError):
            call()
