"""The norm with the residual's addition and its backward pass on the GPU, through the package,
against oracle/block.py in float64.

Tolerances.  h is exact (one rounding of an exact sum).  A value of y before its last rounding
has the float32 errors of s (a sum of at most 64 terms a thread and 12 joins, a square root and a
quotient: under 80 * 2^-24) and of two products, so it is within 2^-17 of the float64 one; bf16
adds half a step, 2^-8 of the value at most; E4M3's half steps are counted by output_errors.
dx = dh + s (a - h s^2 c) is a sum whose terms may cancel: float32 errors count relative to the
terms' sizes (2^-17 of |dh| + s (|a| + |h| s^2 mean|a h|)), and the result is rounded to bf16.
dw is a float32 sum: its errors count relative to the sum of its terms' sizes, at most 64 + 32
additions deep after at most m / 512 + 1 in a row, under 2^-15 for the rows here."""
import numpy as np
import pytest
import torch

from oracle import block as ob
from tests.helpers import DEV, bf16_bits_of, to_dev

pytestmark = pytest.mark.gpu

ql = pytest.importorskip("quantized_linear_layers_block_amd")

EPS = 1e-6
F32 = 2.0 ** -17
BF16 = 2.0 ** -8


def _bits(g, shape, std=1.0):
    return (np.ascontiguousarray((g.normal(size=shape) * std).astype(np.float32)).view(np.uint32) >> 16).astype(np.uint16)


def _f64(t):
    return ob._f64(bf16_bits_of(t))


# k: one unit of 8, partial waves, one workgroup, three units a thread, a thousand threads; m: one
# row, odd rows, and more rows than the grid holds for the wave-a-row variants
SIZES = [(1, 8), (3, 128), (5, 264), (1, 4096), (2, 3584), (7, 5120), (3, 8192), (2, 16384), (2, 24576), (1, 65536),
         (1025, 520), (1500, 1024), (2049, 2048), (20001, 128), (9001, 640)]


@pytest.mark.parametrize("m,k", SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_bf16(m, k, residual):
    print(f"norm m={m} k={k} residual={residual}", flush=True)
    g = np.random.default_rng(m * 7 + k)
    x, r, w = _bits(g, (m, k)), _bits(g, (m, k), 3.0), _bits(g, (k,))
    if residual:
        y, h = ql.rms_norm(to_dev(x), to_dev(w), EPS, residual=to_dev(r))
        hb = ob.add_residual(x, r)
        assert np.array_equal(bf16_bits_of(h), hb)
    else:
        y, hb = ql.rms_norm(to_dev(x), to_dev(w), EPS), x
    ref = ob.rms_norm(ob._f64(hb), ob._f64(w), EPS)
    assert (np.abs(_f64(y) - ref) <= np.abs(ref) * (BF16 + F32)).all()


@pytest.mark.parametrize("m,k", [s for s in SIZES if s[1] % 128 == 0])
@pytest.mark.parametrize("pow2", [False, True])
def test_norm_fp8(m, k, pow2):
    print(f"norm fp8 m={m} k={k} pow2={pow2}", flush=True)
    g = np.random.default_rng(m * 11 + k)
    # segments of very different sizes, one of zeros
    x = (g.normal(size=(m, k // 128, 128)) * 10.0 ** g.integers(-8, 3, size=(m, k // 128, 1))).astype(np.float32)
    x[m // 2, k // 256] = 0
    x = (np.ascontiguousarray(x.reshape(m, k)).view(np.uint32) >> 16).astype(np.uint16)
    w = _bits(g, (k,))
    y = torch.empty((m, k), dtype=torch.bfloat16, device=DEV)
    yq, sy = ql.rms_norm_fp8(to_dev(x), to_dev(w), EPS, pow2=pow2, y=y)
    ref = ob.rms_norm(ob._f64(x), ob._f64(w), EPS)
    assert max(ob.output_errors(yq.cpu().numpy(), sy.cpu().numpy(), ref, F32)) <= 1.0
    assert (np.abs(_f64(y) - ref) <= np.abs(ref) * (BF16 + F32)).all()
    # the same bits without y, and with a residual of zeros
    aq, sa = ql.rms_norm_fp8(to_dev(x), to_dev(w), EPS, pow2=pow2)
    bq, sb, h = ql.rms_norm_fp8(to_dev(x), to_dev(w), EPS, pow2=pow2, residual=torch.zeros_like(y))
    assert torch.equal(aq, yq) and torch.equal(sa, sy) and torch.equal(sb, sy)
    assert torch.equal(bq & 0x7F, yq & 0x7F)   # (the sum of -0 and 0 is 0)


def _check_backward(dx, dw, dy, h, w, dh, eps=EPS):
    dy, h, w = ob._f64(dy), ob._f64(h), ob._f64(w)
    dh = None if dh is None else ob._f64(dh)
    rdx, rdw = ob.rms_norm_backward(dy, h, w, eps, dh)
    s = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    size = s * (np.abs(dy * w) + np.abs(h) * s * s * np.abs(dy * w * h).mean(1, keepdims=True))
    size = size if dh is None else size + np.abs(dh)
    assert (np.abs(_f64(dx) - rdx) <= np.abs(rdx) * BF16 + size * F32 * 2).all()
    if dw is not None:
        assert dw.dtype == torch.float32
        assert (np.abs(dw.cpu().numpy() - rdw) <= np.abs(dy * h * s).sum(0) * 2.0 ** -15).all()


@pytest.mark.parametrize("m,k", SIZES)
@pytest.mark.parametrize("with_dh", [False, True])
def test_norm_backward(m, k, with_dh):
    print(f"norm backward m={m} k={k} dh={with_dh}", flush=True)
    g = np.random.default_rng(m * 13 + k)
    h, dy, w, dh = _bits(g, (m, k), 2.0), _bits(g, (m, k)), _bits(g, (k,)), _bits(g, (m, k))
    args = [to_dev(dy), to_dev(h), to_dev(w), EPS]
    d = to_dev(dh) if with_dh else None
    dx, dw = ql.rms_norm_backward(*args, dh=d)
    _check_backward(dx, dw, dy, h, w, dh if with_dh else None)
    # bitwise the same again, without dweight, and in place of dh or dy
    ws = torch.full((ql.binding.qlinear_rms_norm_backward_workspace(m, k),), 255, dtype=torch.uint8, device=DEV)
    again = ql.rms_norm_backward(*args, dh=d, ws=ws)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    alone = ql.rms_norm_backward(*args, dh=d, need_dweight=False)
    assert alone[1] is None and torch.equal(alone[0], dx)
    over = d.clone() if with_dh else args[0].clone()
    if with_dh:
        ql.rms_norm_backward(*args, dh=over, dx=over)
    else:
        ql.rms_norm_backward(over, *args[1:], dx=over)
    assert torch.equal(over, dx)


@pytest.mark.parametrize("m,k", [(5, 256), (1300, 384), (3, 4096)])
def test_norm_strides_and_in_place(m, k):
    print(f"norm strides m={m} k={k}", flush=True)
    g = np.random.default_rng(k)
    x, r, w, dy = (to_dev(_bits(g, s)) for s in ((m, k), (m, k), (k,), (m, k)))
    y0, h0 = ql.rms_norm(x, w, EPS, residual=r)
    wide = torch.zeros((m, 2 * k + 16), dtype=torch.bfloat16, device=DEV)
    part = wide[:, 8:8 + k]
    part.copy_(x)
    rows = torch.zeros((m, 3, k), dtype=torch.bfloat16, device=DEV)
    rows[:, 1] = r
    before = rows.clone()
    res = rows[:, 1]
    y, h = ql.rms_norm(part, w, EPS, residual=res, h=res)   # the stream updated in place
    assert h is res and torch.equal(h, h0) and torch.equal(y, y0)
    assert torch.equal(rows[:, 0], before[:, 0]) and torch.equal(rows[:, 2], before[:, 2])
    assert torch.equal(part, x) and not wide[:, :8].any() and not wide[:, 8 + k:].any()
    y, h = ql.rms_norm(part, w, EPS, residual=r, h=part)
    assert torch.equal(part, h0) and torch.equal(y, y0)
    dx0, dw0 = ql.rms_norm_backward(dy, h0, w, EPS, dh=r)
    out = torch.zeros((m, k + 24), dtype=torch.bfloat16, device=DEV)
    dx, dw = ql.rms_norm_backward(dy, part, w, EPS, dh=r, dx=out[:, :k])
    assert torch.equal(dx, dx0) and torch.equal(dw, dw0) and not out[:, k:].any()


def test_norm_special_values():
    print("norm special values", flush=True)
    k = 256
    g = np.random.default_rng(5)
    x = _bits(g, (8, k))
    x[1] = 0                                     # a row of zeros
    x[2] = _bits(g, (k,), 1e30)                  # squares beyond float32
    x[3] = _bits(g, (k,), 1e-30)                 # squares below it: eps alone counts
    x[4, 130] = 0x7F80                           # Inf
    x[5, 3] = 0x7FC0                             # NaN
    x[6] = 0x7F7F                                # the largest bf16
    x[7] = _bits(g, (k,), 1e-39)                 # subnormal
    w = _bits(g, (k,))
    with np.errstate(all="ignore"):
        ref = ob.rms_norm(ob._f64(x), ob._f64(w), EPS)
    for pow2 in (False, True):
        y = torch.empty((8, k), dtype=torch.bfloat16, device=DEV)
        yq, sy = ql.rms_norm_fp8(to_dev(x), to_dev(w), EPS, pow2=pow2, y=y)
        good = [0, 1, 2, 3, 6, 7]
        # (2^-134: half of bf16's smallest step, for values below its normal range)
        assert (np.abs(_f64(y)[good] - ref[good]) <= np.abs(ref[good]) * (BF16 + F32) + 2.0 ** -134).all()
        q, s = yq.cpu().numpy(), sy.cpu().numpy()
        assert max(ob.output_errors(q[good], s[good], ref[good], F32)) <= 1.0
        assert not torch.isfinite(y[5]).any() and torch.isnan(y[4, 130])
        nan = (lambda t: t == 0xFF) if pow2 else np.isnan
        assert nan(s[5]).all() and nan(s[4, 1])
    dy = to_dev(_bits(g, (8, k)))
    dx, _ = ql.rms_norm_backward(dy, to_dev(x), to_dev(w), EPS)
    rdx, _ = ob.rms_norm_backward(ob._f64(bf16_bits_of(dy))[good], ob._f64(x)[good], ob._f64(w), EPS)
    got = _f64(dx)[good]
    top = np.abs(rdx).max(1, keepdims=True)
    assert (np.abs(got - rdx) <= np.abs(rdx) * BF16 + top * 2.0 ** -12 + 2.0 ** -134).all()
    assert torch.isnan(dx[5]).any()


def test_norm_border_of_a_power_of_two():
    # the segment's largest value on 448 * 2^e exactly, and one step of float32 over it: rows whose norm is the identity
    k = 128
    x = np.zeros((1, k), np.uint16)
    x[0, :] = 0x3F80
    w = np.zeros(k, np.float32)
    w[3] = 448.0
    wb = (w.view(np.uint32) >> 16).astype(np.uint16)
    yq, sy = ql.rms_norm_fp8(to_dev(x), to_dev(wb), 2.0 ** -40, pow2=True)
    assert int(sy[0, 0]) == 127 and int(yq[0, 3]) == 0x7E and not yq[0, :3].any()
    w[3] = 450.0
    wb = (w.view(np.uint32) >> 16).astype(np.uint16)
    yq, sy = ql.rms_norm_fp8(to_dev(x), to_dev(wb), 2.0 ** -40, pow2=True)
    assert int(sy[0, 0]) == 128 and int(yq[0, 3]) == 0x76   # 224


def test_norm_streams_and_graph():
    print("norm graph", flush=True)
    m, k = 300, 1024
    g = np.random.default_rng(8)
    x, r, w, dy = (to_dev(_bits(g, s)) for s in ((m, k), (m, k), (k,), (m, k)))
    nb = ql.binding.qlinear_rms_norm_backward_workspace(m, k)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)

    def step():
        yq, sy, h = ql.rms_norm_fp8(x, w, EPS, residual=r)
        dx, dw = ql.rms_norm_backward(dy, h, w, EPS, dh=r, ws=ws)
        return yq, sy, h, dx, dw

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        x.copy_(to_dev(_bits(np.random.default_rng(20 + i), (m, k))))
        want = [t.clone() for t in step()]
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, want)), i


# rows over several waves (256 and 1024 threads), several rows a workgroup: up to 2048 (or 512) workgroups forward, 256 or
# 512 backward
@pytest.mark.parametrize("m,k", [(1100, 2560), (2100, 4096), (700, 8192), (2600, 2304), (1600, 8320), (1200, 16512)])
def test_norm_rows_beyond_float32_among_others(m, k):
    """Rows whose squares pass float32 take more sums than the others: both kinds in turn in one workgroup."""
    print(f"norm mixed rows m={m} k={k}", flush=True)
    g = np.random.default_rng(m + k)
    x, w, dy, dh = _bits(g, (m, k), 2.0), _bits(g, (k,)), _bits(g, (m, k)), _bits(g, (m, k))
    far = g.random(m) < 0.4
    x[far] = _bits(g, (int(far.sum()), k), 1e30)
    xd, wd = to_dev(x), to_dev(w)
    y = torch.empty((m, k), dtype=torch.bfloat16, device=DEV)
    yq, sy = ql.rms_norm_fp8(xd, wd, EPS, y=y)
    ref = ob.rms_norm(ob._f64(x), ob._f64(w), EPS)
    assert (np.abs(_f64(y) - ref) <= np.abs(ref) * (BF16 + F32)).all()
    assert max(ob.output_errors(yq.cpu().numpy(), sy.cpu().numpy(), ref, F32)) <= 1.0
    for d in (None, dh):
        dx, dw = ql.rms_norm_backward(to_dev(dy), xd, wd, EPS, dh=None if d is None else to_dev(d))
        _check_backward(dx, dw, dy, x, w, d)


@pytest.mark.parametrize("m,k", [(300, 256), (2100, 1024), (1100, 2560), (600, 8320), (5, 16640)])
@pytest.mark.parametrize("eps", [2.0 ** -149, 2.0 ** -140, 2.0 ** -100, 1e-6])
def test_norm_sums_out_of_range(m, k, eps):
    """An eps below float32's usual numbers with rows as small, whose squares are subnormal or 0; gradients
    whose products with h pass float32, beside usual rows."""
    print(f"norm sums out of range m={m} k={k} eps={eps}", flush=True)
    g = np.random.default_rng(m + k)
    size = g.integers(-85, 40, size=(m, 1))
    x, w = g.normal(size=(m, k)) * 2.0 ** size, _bits(g, (k,))
    dy = g.normal(size=(m, k)) * 2.0 ** np.where(size > 10, g.integers(70, 105, size=(m, 1)), 0)
    x, dy = ((np.ascontiguousarray(t.astype(np.float32)).view(np.uint32) >> 16).astype(np.uint16) for t in (x, dy))
    y = ql.rms_norm(to_dev(x), to_dev(w), eps)
    ref = ob.rms_norm(ob._f64(x), ob._f64(w), eps)
    assert (np.abs(_f64(y) - ref) <= np.abs(ref) * (BF16 + F32) + 2.0 ** -134).all()
    for d in (None, _bits(g, (m, k))):
        dx, dw = ql.rms_norm_backward(to_dev(dy), to_dev(x), to_dev(w), eps, dh=None if d is None else to_dev(d))
        _check_backward(dx, dw, dy, x, w, d, eps)
