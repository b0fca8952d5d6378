"""What stands around the quantized linear layers of a decoder block, as plain float64
definitions: the root-mean-square norm with the residual's addition, the gated feed-forward
block, the 1x128 output quantization of both, and their backward passes.

Source: the mexc.co NeMo RL FP8 page, section "De technische doorbraak": the linear layers take
E4M3 activations with a scale for each 1x128 segment, while norms and nonlinearities stay in
higher precision; the rapidrecap.app Jet-RL summary, "Key Points": FP8 forward, BF16 backward.
The pages state no formula: these are the usual definitions,

    h = bf16(x + residual)      y = h / sqrt(mean(h^2) + eps) * weight
    g = x Wg^T, u = x Wu^T      h = g / (1 + exp(-g)) * u

and their derivatives, every quantization taken as the identity.
"""

import numpy as np

from . import fp8 as _fp8
from .codecs import bf16_bits_to_f32, f32_to_bf16_bits_rne


def _f64(bits):
    return bf16_bits_to_f32(np.asarray(bits, np.uint16)).astype(np.float64)


def add_residual(x_bits, r_bits):
    """bf16 bits of x + r, rounded once (the sum of two bf16 numbers in float32 is rounded to
    bf16 as the exact sum is: float32 keeps 24 bits, which is over twice bf16's 8 plus 2)."""
    return f32_to_bf16_bits_rne(bf16_bits_to_f32(x_bits) + bf16_bits_to_f32(r_bits))


def rms_norm(h, w, eps):
    """y float64 of rows h [m, k] and weight w [k]."""
    h = np.asarray(h, np.float64)
    return h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * np.asarray(w, np.float64)


def rms_norm_backward(dy, h, w, eps, dh=None):
    """(dx [m, k], dw [k])."""
    dy, h, w = (np.asarray(t, np.float64) for t in (dy, h, w))
    s = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    a = dy * w
    dx = s * a - h * s ** 3 * (a * h).mean(1, keepdims=True)
    if dh is not None:
        dx = dx + dh
    return dx, (dy * h * s).sum(0)


def sigmoid(g):
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def gated_forward(x, wg, wu):
    """(h, g, u) float64 of dequantized activations [m, k] and weights [n, k]."""
    g, u = x @ wg.T, x @ wu.T
    return g * sigmoid(g) * u, g, u


def gated_backward(dh, g, u, x, wg, wu):
    """(dx [m, k], dwg [n, k], dwu [n, k])."""
    s = sigmoid(g)
    dg = dh * u * (s + g * s * (1.0 - s))
    du = dh * g * s
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x


def act_values(codes, scales):
    """float64 values of E4M3 activations with float32 scales or E8M0 bytes."""
    scales = np.asarray(scales)
    return _fp8.dequantize_act(codes, _fp8.e8m0_decode(scales) if scales.dtype == np.uint8 else scales)


def weight_values(codes, scales):
    scales = np.asarray(scales)
    return _fp8.dequantize_weight(codes, _fp8.e8m0_decode(scales) if scales.dtype == np.uint8 else scales)


def output_errors(codes, scales, y, tol):
    """How E4M3 codes and their segment scales miss the finite float64 values y [m, k], given that
    the quantized values may be off by `tol` relative to each segment's largest value: (worst
    scale, worst element), each in units of what is allowed, so both are at most 1 where all is
    right.  A code or a scale that is not a number is off by infinity.

    A float32 scale is amax / 448 within tol.  A power of two is the smallest 2^e with
    amax <= 448 2^e, where a rounding may go either way within tol of that border.  An element
    is off by at most half a step of E4M3 of its scale: 2^-4 of its value, or 2^-10 of the scale
    below the normal range, plus tol of the segment's largest value.  A segment of zeros has the
    scale 0 (1 as a power of two) and codes of zero, whatever its tol, which is relative to nothing."""
    m, k = y.shape
    seg = np.asarray(y, np.float64).reshape(m, k // 128, 128)
    amax = np.abs(seg).max(2)
    tol = np.where(amax > 0, tol, 0.0)
    e8m0 = scales.dtype == np.uint8
    s = _fp8.e8m0_decode(scales) if e8m0 else np.asarray(scales, np.float64)
    if e8m0:
        low = np.where((s > 2.0 ** -127) & (amax > 0), amax <= 448.0 * (s / 2) * (1 - tol), False)
        bad = np.where(amax > 0, (amax > 448.0 * s * (1 + tol)) | low, s != 1.0)
        off = np.where(bad, np.inf, 0.0)
        lost = np.asarray(scales) == 0xFF
    else:
        off = np.abs(s - amax / 448.0)
        off = np.where(amax > 0, off / (np.maximum(amax / 448.0 * tol, 2.0 ** -150)), np.where(s == 0, 0, np.inf))
        lost = ~np.isfinite(s)
    worst_scale = np.where(lost | np.isnan(off), np.inf, off).max()
    with np.errstate(invalid="ignore"):
        v = act_values(codes, scales).reshape(seg.shape)
        allowed = np.maximum(np.abs(seg) * 2.0 ** -4, s[..., None] * 2.0 ** -10) + (2 * tol * amax)[..., None] + 2.0 ** -140
        off = np.abs(v - seg) / allowed
    return float(worst_scale), float(np.where(np.isnan(off) | lost[..., None], np.inf, off).max())
