"""NVFP4 KV cache: keys and values as E2M1 codes with an E4M3 scale for 16 elements and one
power-of-two scale for each cached row, and attention over what is held.

The mexc.co page "NVIDIA NeMo RL behaalt 48% snelheidswinst met end-to-end
FP8-precisietraining" (section "Praktische prestatiewinsten") takes the KV cache and attention
to FP8; this is the 4-bit format of the QeRL pages at the same place.  Readings:

* row scale    2^e, e the smallest integer with amax_row <= 2688 * 2^e (2688 = 6 * 448),
  clamped to [-100, 117]; -100 for a zero row;
* block scale  E4M3_RNE(fl32(amax_block * 2^-e / 6));
* code         sign | E2M1_RNE(|x| * 2^-e / scale), magnitude 0 where the scale is 0;
* value        E2M1 * E4M3 * 2^e, exact;
* a token with Inf or NaN in its key or value row of a head: key scale bytes 0xFF, codes and
  value scales 0, e = 0, and NaN values in both rows;
* attention    softmax over the tokens a query row sees, zeros and lse -inf for a row that
  sees none.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""
import numpy as np

from .codecs import bf16_bits_to_f32, e2m1_decode, e2m1_encode_magnitude, e4m3_decode, e4m3_encode_magnitude

F32 = np.float32


def encode_rows(x_bits):
    """bf16 bits [R, D] -> codes uint8 [R, D], scale bytes [R, D/16], e [R]; non-finite rows are
    encoded as zero rows (the caller marks them)."""
    x = bf16_bits_to_f32(np.asarray(x_bits, np.uint16)).astype(np.float64)
    x = np.where(np.isfinite(x), x, 0.0)
    r, d = x.shape
    mag = np.abs(x)
    amax = mag.max(axis=1)
    e = np.full(r, -100)
    for i in range(r):   # the definition, by steps of one
        k = -100
        while k < 117 and amax[i] > 2688.0 * 2.0 ** k:
            k += 1
        e[i] = k
    y = mag * np.exp2(-e.astype(np.float64))[:, None]
    blocks = y.reshape(r, d // 16, 16)
    scale = e4m3_encode_magnitude((blocks.max(axis=2).astype(F32) / F32(6.0)).astype(F32))
    s = e4m3_decode(scale)[:, :, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s > 0, blocks / np.where(s > 0, s, 1.0), 0.0)
    code = e2m1_encode_magnitude(q.astype(F32)).reshape(r, d)
    return (code | (np.signbit(x).astype(np.uint8) << 3)).astype(np.uint8), scale.astype(np.uint8), e


def nonfinite_rows(x_bits):
    return ((np.asarray(x_bits, np.uint16) & 0x7FFF) >= 0x7F80).any(axis=-1)


def group_bytes(d):
    return 18 * d + 32


def empty(pages, heads, d, page_size, fill=0):
    return np.full((pages, heads, page_size // 16, group_bytes(d)), fill, np.uint8)


def _addresses(data, slot, head, d):
    pages, heads, per, gb = data.shape
    base = ((slot // (16 * per) * heads + head) * per + slot % (16 * per) // 16) * gb
    t = slot % 16
    p, b = np.arange(d // 2), np.arange(d // 16)
    kc = base + t * (d // 2) + p
    ks = base + 8 * d + t * (d // 16) + b
    ke = base + 9 * d + t
    v = base + 9 * d + 16
    vc = v + t // 4 * 2 * d + p % 16 * (d // 8) + p // 16 * 4 + t % 4
    vs = v + 8 * d + t // 4 * (d // 4) + b % 2 * (d // 8) + b // 2 * 4 + t % 4
    return kc, ks, ke, vc, vs, v + 9 * d + t


def store(data, k_bits, v_bits, slots):
    """k, v bf16 bits [T, H, D] into the cache (in place); slots outside it are skipped."""
    pages, heads, per, gb = data.shape
    flat = data.reshape(-1)
    t, h, d = k_bits.shape
    bad = nonfinite_rows(k_bits) | nonfinite_rows(v_bits)
    enc = [encode_rows(x.reshape(t * h, d)) for x in (k_bits, v_bits)]
    for i, s in enumerate(np.asarray(slots, np.int64)):
        if s < 0 or s >= pages * per * 16:
            continue
        for j in range(h):
            at = _addresses(data, int(s), j, d)
            for side in range(2):
                code, scale, e = (a[i * h + j] for a in enc[side])
                if bad[i, j]:
                    code, scale, e = np.zeros(d, np.uint8), np.full(d // 16, 0 if side else 0xFF, np.uint8), 0
                flat[at[3 * side]] = code[0::2] | (code[1::2] << 4)
                flat[at[3 * side + 1]] = scale
                flat[at[3 * side + 2]] = e + 127


def load(data, slots, d):
    """-> keys and values float64 [T, H, D]; zeros for slots outside the cache."""
    pages, heads, per, gb = data.shape
    flat = data.reshape(-1)
    out = np.zeros((2, len(slots), heads, d))
    for i, s in enumerate(np.asarray(slots, np.int64)):
        if s < 0 or s >= pages * per * 16:
            continue
        for j in range(heads):
            at = _addresses(data, int(s), j, d)
            for side in range(2):
                byte = flat[at[3 * side]]
                code = np.empty(d, np.uint8)
                code[0::2], code[1::2] = byte & 15, byte >> 4
                scale = np.repeat(e4m3_decode(flat[at[3 * side + 1]]), 16)
                out[side, i, j] = e2m1_decode(code) * scale * 2.0 ** (int(flat[at[3 * side + 2]]) - 127)
                if flat[at[1][0]] == 0xFF:
                    out[side, i, j] = np.nan
    return out[0], out[1]


def sequence_slots(table_row, n, page_size):
    """Slots of a sequence's first n tokens (-1 where the page is outside the table's values)."""
    t = np.arange(n)
    return np.asarray(table_row, np.int64)[t // page_size] * page_size + t % page_size


def attention(q, k, v, scale, causal=True, window=0, held=None):
    """q float64 [nq, Hq, D] of one sequence over its n cached k, v float64 [n, H, D] -> out
    [nq, Hq, D], lse [nq, Hq] and the weighted mean of |v| [nq, Hq, D] (for error bounds).
    held [n]: False for tokens that are left out (a bad page)."""
    nq, hq, d = q.shape
    n, h, _ = k.shape
    out, amean = np.zeros((nq, hq, d)), np.zeros((nq, hq, d))
    lse = np.full((nq, hq), -np.inf)
    tok = np.arange(n)
    for i in range(nq):
        pos = n - nq + i if causal else n - 1
        seen = (tok <= pos) & ((tok > pos - window) if window else True)
        if held is not None:
            seen &= held
        if not seen.any():
            continue
        for j in range(hq):
            kk, vv = k[seen, j // (hq // h)], v[seen, j // (hq // h)]
            s = scale * (kk @ q[i, j])
            top = s.max()
            p = np.exp(s - top)
            out[i, j] = p @ vv / p.sum()
            amean[i, j] = p @ np.abs(vv) / p.sum()
            lse[i, j] = top + np.log(p.sum())
    return out, lse, amean
