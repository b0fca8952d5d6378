"""The gated block's backward pass on the GPU, through the package, against oracle/block.py in
float64, and against differences of the forward's definition.

Tolerances.  dg and du are formed in float32 (within 2^-19 of their size: dg's terms s and
g s (1 - s) have opposite signs for g < 0, so its size is |dh u| s (1 + |g| (1 - s))).
  dx: they enter as f16 (2^-11 of a value, or 2^-25 of 2^15 relative to the row's largest, which
  is at least 2^14), weights as f16 of value * f16(scale) (2^-11 each): 3 * 2^-11 + 2^-18 of
  T = |dg| |Wg| + |du| |Wu|, and a row's 2^-39 of its largest dg or du times sum |W|.
  weights: rounded to bf16, 2^-8 of T = |dg|^T |x|.
Float32 sums of Z products in steps of 32 with at most four roundings of 2^-23 each, split and
joined: (Z / 8 + 40) 2^-23 T.  The result is rounded to bf16, 2^-8 of the value.  As these bounds are
for the worst case, the 2-norm of the difference is held to 2^-8 of the result's as well, where no
gradient is a small rest of a large sum."""
import numpy as np
import pytest
import torch

from oracle import block as ob
from tests.helpers import DEV, bf16_bits_of, to_dev
from tests.test_gpu_gated import _codes, _dev, _scales

pytestmark = pytest.mark.gpu

ql = pytest.importorskip("quantized_linear_layers_block_amd")

BF16 = 2.0 ** -8


def _bits(g, shape, std=1.0):
    return (np.ascontiguousarray((g.normal(size=shape) * std).astype(np.float32)).view(np.uint32) >> 16).astype(np.uint16)


def _case(m, n, k, pow2, seed):
    g = np.random.default_rng(seed)
    ws = [(_codes(g, (n, k)), _scales(g, (n // 128, k // 128), pow2, 0.001)) for _ in range(2)]
    dh = _bits(g, (m, n)).astype(np.uint16)
    # tokens whose gradients are far apart in size, and one without any
    rows = np.float32(10.0) ** g.integers(-6, 2, size=(m, 1)).astype(np.float32)
    dh = (np.ascontiguousarray(ob._f64(dh).astype(np.float32) * rows).view(np.uint32) >> 16).astype(np.uint16)
    if m > 2:
        dh[m // 2] = 0
    return ws, dh, _bits(g, (m, 2 * n), 3.0), _bits(g, (m, k))


def _off(got, ref, err):
    """By how much got passes what is allowed, 1 being the limit."""
    d = np.abs(ob._f64(bf16_bits_of(got)) - ref)
    lim = np.abs(ref) * BF16 + err * (1 + BF16) + 2.0 ** -133
    return float((d / lim).max()), float(np.linalg.norm(d) / max(np.linalg.norm(ref), 1e-300))


def _check(ws, dh, gu, x, got):
    n = dh.shape[1]
    dhv, g, u, xv = ob._f64(dh), ob._f64(gu[:, :n]), ob._f64(gu[:, n:]), ob._f64(x)
    wv = [ob.weight_values(*w) for w in ws]
    rdx, rdg, rdu = ob.gated_backward(dhv, g, u, xv, *wv)
    s = ob.sigmoid(g)
    sg, su = np.abs(dhv * u) * s * (1 + np.abs(g) * (1 - s)), np.abs(dhv * g) * s
    m = dh.shape[0]
    aw = [np.abs(w) for w in wv]
    t = sg @ aw[0] + su @ aw[1]
    top = np.maximum(sg.max(1), su.max(1))[:, None]
    e = t * (3 * 2.0 ** -11 + 2.0 ** -17 + (2 * n / 8 + 40) * 2.0 ** -23) + 2.0 ** -39 * top * (aw[0].sum(0) + aw[1].sum(0))
    # (the smallest scales of a column block lose bits as f16: 2^-25 of what the largest is, 32)
    e += 2.0 ** -30 * (sg + su).sum(1, keepdims=True) * np.maximum(aw[0].max(0), aw[1].max(0))
    worst, rel = _off(got[0], rdx, e)
    assert worst <= 1 and rel <= BF16, (worst, rel)
    ax = np.abs(xv)
    for out, ref, size in ((got[1], rdg, sg), (got[2], rdu, su)):
        worst, rel = _off(out, ref, (size.T @ ax) * (BF16 + 2.0 ** -17 + (m / 8 + 40) * 2.0 ** -23))
        assert worst <= 1 and rel <= BF16, (worst, rel)


# m around tiles and steps; n and k with half tiles; depths long enough to be split among workgroups
@pytest.mark.parametrize("m,n,k", [(1, 128, 128), (5, 256, 384), (31, 128, 256), (32, 384, 128), (33, 128, 640), (100, 256, 256),
                                   (255, 128, 128), (256, 640, 512), (257, 128, 384), (600, 384, 256), (2000, 128, 128),
                                   (7, 4224, 128), (3, 8320, 256), (2, 16512, 128), (64, 2176, 512), (2048, 128, 384),
                                   (2111, 256, 128), (40, 2176, 4224), (129, 4224, 2304)])
@pytest.mark.parametrize("pow2", [False, True])
def test_gated_backward(m, n, k, pow2):
    print(f"gated backward m={m} n={n} k={k} pow2={pow2}", flush=True)
    ws, dh, gu, x = _case(m, n, k, pow2, m + 5 * n + k)
    gate, up = [ql.FP8Weight(_dev(c), _dev(s), n, k, pow2) for c, s in ws]
    args = gate, up, to_dev(dh), to_dev(gu), to_dev(x)
    got = ql.gated_backward(*args)
    _check(ws, dh, gu, x, got)
    # the same bits again on a workspace of anything, and each gradient alone
    buf = torch.full((ql.binding.qlinear_gated_backward_workspace(m, n, k),), 255, dtype=torch.uint8, device=DEV)
    assert all(torch.equal(p, q) for p, q in zip(ql.gated_backward(*args, ws=buf), got))
    one = ql.gated_backward(*args[:4], need_dweight=False, ws=buf)
    assert torch.equal(one[0], got[0]) and one[1] is None and one[2] is None
    two = ql.gated_backward(*args, need_dx=False, ws=buf.fill_(255))
    assert two[0] is None and torch.equal(two[1], got[1]) and torch.equal(two[2], got[2])


# thousands of tokens, where dx reads the weights turned beforehand: around the border, ragged rows, half tiles of n and k
@pytest.mark.parametrize("m,n,k", [(2815, 128, 256), (2816, 256, 128), (2911, 128, 384), (4100, 384, 256)])
@pytest.mark.parametrize("pow2", [False, True])
def test_gated_backward_many(m, n, k, pow2):
    test_gated_backward(m, n, k, pow2)


# thousands of tokens: more tiles than a round of the chip (weights turned beforehand), and both products in one round
@pytest.mark.parametrize("m,n,k", [(2816, 256, 6272), (2911, 128, 5760), (4100, 128, 4096), (5000, 512, 512), (1347, 1664, 1920)])
@pytest.mark.parametrize("pow2", [False, True])
def test_gated_backward_plans(m, n, k, pow2):
    test_gated_backward(m, n, k, pow2)


def test_special_values_turned():
    """As test_special_values_many where the weights are turned beforehand."""
    print("gated backward special turned", flush=True)
    m, n, k = 2820, 128, 5888
    ws, dh, gu, x = _case(m, n, k, True, 6)
    gate, up = [ql.FP8Weight(_dev(c), _dev(s), n, k, True) for c, s in ws]
    want = ql.gated_backward(gate, up, to_dev(dh), to_dev(gu), to_dev(x))
    bad = dh.copy()
    bad[2817, 40] = 0x7FC0
    up.codes[7, 5800] = 0x7F
    got = ql.gated_backward(gate, up, to_dev(bad), to_dev(gu), to_dev(x))
    nan = torch.isnan(got[0])
    assert nan[2817].all() and nan[:, 5800].all()
    clean = ~nan
    assert clean.sum() == (m - 1) * (k - 1) and torch.equal(got[0][clean], want[0][clean])


def test_special_values_many():
    """A NaN code of the weights reaches its column of dx, a NaN of dh its row, and nothing else."""
    print("gated backward special many", flush=True)
    m, n, k = 2820, 256, 256
    ws, dh, gu, x = _case(m, n, k, True, 5)
    gate, up = [ql.FP8Weight(_dev(c), _dev(s), n, k, True) for c, s in ws]
    want = ql.gated_backward(gate, up, to_dev(dh), to_dev(gu), to_dev(x))
    _check(ws, dh, gu, x, want)
    bad = dh.copy()
    bad[2817, 40] = 0x7FC0
    up.codes[7, 100] = 0x7F
    got = ql.gated_backward(gate, up, to_dev(bad), to_dev(gu), to_dev(x))
    nan = torch.isnan(got[0])
    assert nan[2817].all() and nan[:, 100].all()
    clean = ~nan
    assert clean.sum() == (m - 1) * (k - 1) and torch.equal(got[0][clean], want[0][clean])
    rows = np.delete(np.arange(n), 40)
    for p, q in zip(got[1:], want[1:]):
        assert torch.isnan(p[40]).all() and torch.equal(p[rows], q[rows])


@pytest.mark.parametrize("pow2", [False, True])
def test_special_values(pow2):
    print(f"gated backward special pow2={pow2}", flush=True)
    m, n, k = 70, 256, 256
    ws, dh, gu, x = _case(m, n, k, pow2, 3)
    gu[3, :n] = 0x42C8       # gates of 100 and -100, the largest and smallest bf16: silu is the gate or 0
    gu[4, :n] = 0xC2C8
    gu[5, :n] = 0x7F7F
    gu[5, n:] = 0x0080
    gu[6, :n] = 0xFF7F
    dh[5:7] = 0x0080         # 2^-126: products stay in range
    gate, up = [ql.FP8Weight(_dev(c), _dev(s), n, k, pow2) for c, s in ws]
    got = ql.gated_backward(gate, up, to_dev(dh), to_dev(gu), to_dev(x))
    assert all(torch.isfinite(t).all() for t in got)
    keep = np.delete(np.arange(m), [5, 6])
    clean = gu.copy()
    clean[5:7] = 0
    dh2 = dh.copy()
    dh2[5:7] = 0
    got2 = ql.gated_backward(gate, up, to_dev(dh2), to_dev(clean), to_dev(x))
    _check(ws, dh2, clean, x, got2)
    assert torch.equal(got[0][keep], got2[0][keep])
    # NaN and Inf reach what they are part of, and nothing else
    bad = dh2.copy()
    bad[9, 17] = 0x7FC0
    got3 = ql.gated_backward(gate, up, to_dev(bad), to_dev(clean), to_dev(x))
    rest = np.delete(np.arange(m), 9)
    assert torch.isnan(got3[0][9]).all() and torch.equal(got3[0][rest], got2[0][rest])
    cols = np.delete(np.arange(n), 17)
    for p, q in zip(got3[1:], got2[1:]):
        assert torch.isnan(p[17]).all() and torch.equal(p[cols], q[cols])
    bx = x.copy()
    bx[m - 1, 5] = 0x7F80    # Inf in the last token, next to the padding
    got4 = ql.gated_backward(gate, up, to_dev(dh2), to_dev(clean), to_dev(bx))
    others = np.delete(np.arange(k), 5)
    for p, q in zip(got4[1:], got2[1:]):
        assert not torch.isfinite(p[:, 5]).any() and torch.equal(p[:, others], q[:, others])
    assert torch.isinf(got4[1][:, 5]).any() or torch.isinf(got4[2][:, 5]).any()


def test_against_differences():
    """The gradients against differences of the forward's float64 definition along directions."""
    print("gated backward differences", flush=True)
    g = np.random.default_rng(8)
    m, n, k = 40, 256, 384
    ws, dh, _, x = _case(m, n, k, False, 12)
    dh = _bits(g, (m, n))
    wv = [ob.weight_values(*w) for w in ws]
    xv = ob._f64(x)
    _, gg, uu = ob.gated_forward(xv, *wv)
    gu = (np.ascontiguousarray(np.concatenate((gg, uu), 1).astype(np.float32)).view(np.uint32) >> 16).astype(np.uint16)
    gate, up = [ql.FP8Weight(_dev(c), _dev(s), n, k, False) for c, s in ws]
    got = [ob._f64(bf16_bits_of(t)) for t in ql.gated_backward(gate, up, to_dev(dh), to_dev(gu), to_dev(x))]
    at = [xv] + wv
    for i in range(3):
        way = got[i] / np.linalg.norm(got[i])          # along the gradient itself: no cancellation
        step = 1e-6 * np.linalg.norm(at[i])
        loss = lambda t: (ob.gated_forward(*[at[j] + t * way if j == i else at[j] for j in range(3)])[0] * ob._f64(dh)).sum()   # noqa: E731
        slope = (loss(step) - loss(-step)) / (2 * step)
        # gu is cut to bf16 (2^-7), and silu' moves by at most |d silu'/dg| <= 1/2 of that times |g|
        assert abs((got[i] * way).sum() - slope) <= 0.03 * abs(slope), i


def test_training_step_of_a_block():
    """norm -> gated block -> its backward -> the norm's backward, as one captured step and eagerly."""
    print("training step", flush=True)
    g = np.random.default_rng(4)
    m, n, k = 90, 384, 256
    x, r, w, dh = (to_dev(_bits(g, s, t)) for s, t in (((m, k), 1.0), ((m, k), 2.0), ((k,), 1.0), ((m, n), 0.1)))
    gate, up = (ql.quantize_fp8_block(to_dev(_bits(g, (n, k), 0.05))) for _ in range(2))
    ws = torch.zeros(ql.binding.qlinear_gated_forward_workspace(m, n, k), dtype=torch.uint8, device=DEV)
    wb = torch.empty(ql.binding.qlinear_gated_backward_workspace(m, n, k), dtype=torch.uint8, device=DEV)
    wn = torch.empty(ql.binding.qlinear_rms_norm_backward_workspace(m, k), dtype=torch.uint8, device=DEV)

    def step():
        y = torch.empty_like(x)
        gu = torch.empty((m, 2 * n), dtype=torch.bfloat16, device=DEV)
        yq, sy, h = ql.rms_norm_fp8(x, w, residual=r, y=y)
        act = ql.gated_forward(gate, up, yq, sy, gu=gu, ws=ws)
        dy, dgate, dup = ql.gated_backward(gate, up, dh, gu, y, ws=wb)
        dx, dw = ql.rms_norm_backward(dy, h, w, dh=r, ws=wn)
        return act, dgate, dup, dx, dw, gu, y, dy

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, first))
    for i in range(3):
        x.copy_(to_dev(_bits(np.random.default_rng(i), (m, k))))
        want = [t.clone() for t in step()]
        wb.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), i
    # the chain against float64 from what each step was given
    f = lambda t: ob._f64(bf16_bits_of(t))   # noqa: E731
    vals = [ob.weight_values(q.codes.cpu().numpy(), q.scales.cpu().numpy()) for q in (gate, up)]
    rdx, rdg, rdu = ob.gated_backward(f(dh), f(got[5][:, :n]), f(got[5][:, n:]), f(got[6]), *vals)
    for p, q in ((got[7], rdx), (got[1], rdg), (got[2], rdu)):
        assert np.linalg.norm(f(p) - q) <= BF16 * np.linalg.norm(q)


@pytest.mark.parametrize("m,n,k", [(2, 256, 384), (130, 2176, 256), (300, 384, 512), (2900, 256, 128)])
def test_two_streams_and_a_graph(m, n, k):
    """Calls side by side on two streams with a workspace each, and a captured one between eager ones."""
    print(f"gated backward streams m={m} n={n} k={k}", flush=True)
    ws, dh, gu, x = _case(m, n, k, True, 31)
    gate, up = [ql.FP8Weight(_dev(c), _dev(s), n, k, True) for c, s in ws]
    dev = to_dev(dh), to_dev(gu), to_dev(x)
    want = ql.gated_backward(gate, up, *dev)
    size = ql.binding.qlinear_gated_backward_workspace(m, n, k)
    spaces = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    out = []
    for _ in range(4):
        for s in range(2):
            with torch.cuda.stream(streams[s]):
                out.append(ql.gated_backward(gate, up, *dev, ws=spaces[s]))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for got in out for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ql.gated_backward(gate, up, *dev, ws=spaces[0])
    for i in range(3):
        dev[0].copy_(to_dev(_bits(np.random.default_rng(i), (m, n), 0.1)))
        want = ql.gated_backward(gate, up, *dev, ws=spaces[1])
        spaces[0].fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), i


# dx's kernels: tiles of 128 and of 256 rows, alone and beside the weights' gradients, weights turned beforehand
@pytest.mark.parametrize("m,n,k", [(70, 256, 256), (300, 384, 512), (200, 8320, 640), (2900, 256, 6272)])
@pytest.mark.parametrize("pow2", [False, True])
def test_rows_of_any_size(m, n, k, pow2):
    """Gradients from 2^-100 to 2^112 a row: a row's factor alone passes float32 where dx does not."""
    print(f"gated backward rows of any size m={m} n={n} k={k} pow2={pow2}", flush=True)
    ws, _, gu, x = _case(m, n, k, pow2, m + n)
    g = np.random.default_rng(m)
    dh = np.ldexp(g.normal(size=(m, n)), g.integers(-100, 113, size=(m, 1))).astype(np.float32)
    dh = (np.ascontiguousarray(dh).view(np.uint32) >> 16).astype(np.uint16)
    gate, up = [ql.FP8Weight(_dev(c), _dev(s), n, k, pow2) for c, s in ws]
    got = ql.gated_backward(gate, up, to_dev(dh), to_dev(gu), to_dev(x))
    _check(ws, dh, gu, x, got)
    one = ql.gated_backward(gate, up, to_dev(dh), to_dev(gu), need_dweight=False)[0]
    assert torch.equal(one, got[0])


@pytest.mark.parametrize("m,n,k", [(60, 256, 128), (130, 4224, 128), (40, 8320, 256), (20, 16512, 128)])
@pytest.mark.parametrize("pow2", [False, True])
def test_gates_far_below_zero(m, n, k, pow2):
    """Rows of gates down to -160 with dh and u so large that dg is of usual size: exp(g) is below float32's
    smallest number, dh u above its largest."""
    print(f"gated backward far gates m={m} n={n} k={k} pow2={pow2}", flush=True)
    ws, _, _, x = _case(m, n, k, pow2, m + n)
    g = np.random.default_rng(m)
    level = g.uniform(-160, 0, size=(m, 1))
    gates = level + g.normal(size=(m, n))
    room = -level / np.log(2)                                  # dh u of 2^room and some
    a = np.clip(room * g.uniform(0.4, 0.6, size=(m, 1)), room - 120, 120)
    dh, u = g.normal(size=(m, n)) * 2 ** a, g.normal(size=(m, n)) * 2 ** (room - a)
    dh, gu = ((np.ascontiguousarray(t.astype(np.float32)).view(np.uint32) >> 16).astype(np.uint16)
              for t in (dh, np.concatenate((gates, u), 1)))
    with np.errstate(over="ignore"):
        assert np.isinf(ob._f64(dh).astype(np.float32) * ob._f64(gu[:, n:]).astype(np.float32)).any()
    gate, up = [ql.FP8Weight(_dev(c), _dev(s), n, k, pow2) for c, s in ws]
    got = ql.gated_backward(gate, up, to_dev(dh), to_dev(gu), to_dev(x))
    _check(ws, dh, gu, x, got)


# more tiles than a round of the chip: the last count of tokens whose weights dx turns as it reads them, the first whose
# weights are turned beforehand, and one of the latter with parts of dx; K with half tiles
@pytest.mark.parametrize("m,n,k", [(2815, 128, 5888), (2816, 128, 5888), (2977, 384, 5504)])
@pytest.mark.parametrize("pow2", [False, True])
def test_gated_backward_turned_border(m, n, k, pow2):
    test_gated_backward(m, n, k, pow2)


# the plans with a launch for each product: weights turned beforehand (the turned copy lies in the workspace), and weights'
# gradients of few tokens two workgroups a CU
@pytest.mark.parametrize("m,n,k", [(2820, 128, 5888), (40, 2176, 4224)])
def test_two_streams_and_a_graph_apart(m, n, k):
    test_two_streams_and_a_graph(m, n, k)


@pytest.mark.parametrize("m,n,k", [(40, 256, 128), (20, 16512, 128)])
def test_gates_beyond_every_product(m, n, k):
    """Gates from -200 to -400 beside dh and u of 2^124: dg goes from 2^-30 to nothing, and so does what follows.

    du is below 2^125 400 exp(-195) = 2^-147, so a weight gradient of up is below 2^-147 m max|x| < 2^-139:
    nothing but 0 is as near in bf16, whose least number is 2^-133, and so it is no part of _check, which holds
    2-norms to each other.  dx and the gate's gradient are held to the bounds above."""
    print(f"gated backward gates beyond m={m} n={n} k={k}", flush=True)
    ws, _, _, x = _case(m, n, k, False, m + n)
    g = np.random.default_rng(m)
    gates = np.linspace(-200, -400, m)[:, None] + g.normal(size=(m, n))
    dh, u = (g.choice([-1.0, 1.0], size=(m, n)) * 2.0 ** 124 * g.uniform(1, 2, size=(m, n)) for _ in range(2))
    dh, gu = ((np.ascontiguousarray(t.astype(np.float32)).view(np.uint32) >> 16).astype(np.uint16)
              for t in (dh, np.concatenate((gates, u), 1)))
    gate, up = [ql.FP8Weight(_dev(c), _dev(s), n, k, False) for c, s in ws]
    dx, dgate, dup = ql.gated_backward(gate, up, to_dev(dh), to_dev(gu), to_dev(x))
    dhv, gv, uv, xv = ob._f64(dh), ob._f64(gu[:, :n]), ob._f64(gu[:, n:]), ob._f64(x)
    wv = [ob.weight_values(*w) for w in ws]
    rdx, rdg, _ = ob.gated_backward(dhv, gv, uv, xv, *wv)
    assert np.abs(xv).max() * m < 2.0 ** 8 and not dup.any()
    sg, su = np.abs(dhv * uv * np.exp(gv) * (1 + gv)), np.abs(dhv * gv * np.exp(gv))
    aw = [np.abs(w) for w in wv]
    top = np.maximum(sg.max(1), su.max(1))[:, None]
    e = (sg @ aw[0] + su @ aw[1]) * (3 * 2.0 ** -11 + 2.0 ** -17 + (2 * n / 8 + 40) * 2.0 ** -23)
    e += 2.0 ** -39 * top * (aw[0].sum(0) + aw[1].sum(0))
    e += 2.0 ** -30 * (sg + su).sum(1, keepdims=True) * np.maximum(aw[0].max(0), aw[1].max(0))
    assert _off(dx, rdx, e)[0] <= 1
    assert _off(dgate, rdg, (sg.T @ np.abs(xv)) * (BF16 + 2.0 ** -17 + (m / 8 + 40) * 2.0 ** -23))[0] <= 1
