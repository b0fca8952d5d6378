"""The float64 definitions of oracle/block.py against differences of themselves, exact cases and
hand-made values: what the GPU tests of the norm and the gated block compare with."""
import numpy as np
import pytest

from oracle import block as ob, fp8 as ofp8


def _slope(f, at, way, step=1e-5):
    return (f(at + step * way) - f(at - step * way)) / (2 * step)


def test_norm_by_hand():
    h = np.array([[3.0, 4.0], [0.0, 0.0]])
    y = ob.rms_norm(h, np.array([1.0, 2.0]), 1e-300)
    s = np.sqrt(12.5)
    assert np.allclose(y, [[3 / s, 8 / s], [0, 0]], rtol=1e-15)


@pytest.mark.parametrize("seed", [1, 2])
def test_norm_gradients_are_the_slopes(seed):
    g = np.random.default_rng(seed)
    h, w, dy, dh = g.normal(size=(5, 24)), g.normal(size=24), g.normal(size=(5, 24)), g.normal(size=(5, 24))
    dx, dw = ob.rms_norm_backward(dy, h, w, 0.3, dh)
    way, wayw = g.normal(size=h.shape), g.normal(size=24)
    assert np.isclose((dx * way).sum(), _slope(lambda t: (ob.rms_norm(t, w, 0.3) * dy + t * dh).sum(), h, way), rtol=1e-8)
    assert np.isclose((dw * wayw).sum(), _slope(lambda t: (ob.rms_norm(h, t, 0.3) * dy).sum(), w, wayw), rtol=1e-8)


@pytest.mark.parametrize("seed", [3, 4])
def test_gated_gradients_are_the_slopes(seed):
    g = np.random.default_rng(seed)
    x, wg, wu = g.normal(size=(4, 6)), g.normal(size=(7, 6)), g.normal(size=(7, 6))
    dh = g.normal(size=(4, 7))
    _, gg, uu = ob.gated_forward(x, wg, wu)
    grads = ob.gated_backward(dh, gg, uu, x, wg, wu)
    loss = lambda *t: (ob.gated_forward(*t)[0] * dh).sum()   # noqa: E731
    for i, got in enumerate(grads):
        way = g.normal(size=got.shape)
        at = [x, wg, wu]
        f = lambda t: loss(*[t if j == i else at[j] for j in range(3)])   # noqa: E731
        assert np.isclose((got * way).sum(), _slope(f, at[i], way), rtol=1e-7), i


def test_sigmoid_far_out():
    assert np.array_equal(ob.sigmoid(np.array([0.0, 1000.0, -1000.0])), [0.5, 1.0, 0.0])


@pytest.mark.parametrize("pow2", [False, True])
def test_output_errors_accept_the_quantizer_and_see_a_wrong_code(pow2):
    g = np.random.default_rng(9)
    bits = (g.normal(size=(6, 256)) * 10.0 ** g.integers(-6, 4, size=(6, 1))).astype(np.float32)
    bits[2, :128] = 0
    bits = (bits.view(np.uint32) >> 16).astype(np.uint16)
    y = ob._f64(bits)
    codes, s = (ofp8.quantize_act_pow2 if pow2 else ofp8.quantize_act)(bits)
    assert max(ob.output_errors(codes, s, y, 2.0 ** -22)) <= 1.0
    wrong = codes.copy()
    wrong[4, 200] ^= 2
    assert ob.output_errors(wrong, s, y, 2.0 ** -22)[1] > 1.0
    off = s.copy()
    off[1, 1] = off[1, 1] + 1 if pow2 else off[1, 1] * np.float32(1.001)
    assert ob.output_errors(codes, off, y, 2.0 ** -22)[0] > 1.0


@pytest.mark.parametrize("pow2", [False, True])
def test_output_errors_see_what_is_not_a_number(pow2):
    g = np.random.default_rng(10)
    bits = (g.normal(size=(5, 384)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    bits[3, 128:256] = 0
    y = ob._f64(bits)
    codes, s = (ofp8.quantize_act_pow2 if pow2 else ofp8.quantize_act)(bits)
    # a tolerance relative to the largest value of a segment of zeros is not a number: the segment is held to zeros
    tol = np.full((5, 3), 2.0 ** -22)
    tol[3, 1] = np.nan
    assert max(ob.output_errors(codes, s, y, tol)) <= 1.0
    for where in ((2, 200), (3, 140), slice(None)):
        for code in (0x7F, 0xFF):
            wrong = codes.copy()
            wrong[where] = code
            assert max(ob.output_errors(wrong, s, y, tol)) == np.inf, (where, code)
    for where in ((2, 1), (3, 1), slice(None)):
        for scale in ((255,) if pow2 else (np.nan, np.inf)):
            wrong = s.copy()
            wrong[where] = scale
            assert max(ob.output_errors(codes, wrong, y, tol)) == np.inf, (where, scale)
    # values where there are none
    wrong, off = codes.copy(), s.copy()
    wrong[3, 130], off[3, 1] = 1, 127 if pow2 else 1.0
    assert max(ob.output_errors(wrong, off, y, tol)) > 1.0
