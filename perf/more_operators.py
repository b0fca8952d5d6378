"""The operators around the FP8 linear layers of a decoder block, as cases to measure: the
root-mean-square norm with the residual's addition and an output in 8 bits, its backward pass,
the gated feed-forward block on FP8 weights, and its backward pass.

norm        h = bf16(x + r), y = h / sqrt(mean(h^2) + eps) * w; y in bf16, or (with a format) as
            E4M3 codes with one scale for 128 columns: float32 amax / 448, or ("pow2") 2^e with
            the smallest e for which amax <= 448 * 2^e
norm_bwd    from dy and the gradient dh that arrives beside the norm: the gradient of h, and dw
gated       g = x Wg^T, u = x Wu^T, h = g / (1 + exp(-g)) * u from E4M3 activations (scales for
            128 columns) and E4M3 weights (scales for 128 x 128); h in bf16 or as codes with scales;
            in training g and u in bf16 too, side by side
gated_bwd   from dh, g and u: dx through both weights, and both weights' gradients
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------------------------- cases

def _norm(name, m, k, fmt="bf16", residual=True, keep_y=False):
    c = dict(op="norm", m=m, k=k, fmt=fmt, residual=residual, keep_y=keep_y)
    return dict(name=name, **c) if name else c


def _norm_bwd(name, m, k, dh=True, dw=True):
    c = dict(op="norm_bwd", m=m, k=k, dh=dh, dw=dw)
    return dict(name=name, **c) if name else c


def _gated(name, m, n, k, fmt, quant=True, train=False):
    c = dict(op="gated", m=m, n=n, k=k, fmt=fmt, quant=quant, train=train)
    return dict(name=name, **c) if name else c


def _gated_bwd(name, m, n, k, fmt):
    c = dict(op="gated_bwd", m=m, n=n, k=k, fmt=fmt)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one user's next token before the FP8 projections of an 8B-class layer: latency alone
        _norm("norm_1x4096_fp8", 1, 4096, "fp8"),
        # a rollout batch of 256 on a 32B-class layer whose projections take bf16
        _norm("norm_256x5120_bf16", 256, 5120),
        # an odd number of prompt tokens of a 7B-class layer, power-of-two scales, no residual yet
        _norm("norm_1777x3584_pow2", 1777, 3584, "pow2", residual=False),
        # a training batch of 8192 tokens: 8 bits for the forward, bf16 kept for the weight gradients
        _norm("norm_8192x4096_fp8_train", 8192, 4096, "fp8", keep_y=True),
        # the gradient of a short batch, odd sizes
        _norm_bwd("norm_bwd_333x3584", 333, 3584),
        # the gradient of a large training batch on a 32B-class layer
        _norm_bwd("norm_bwd_16384x5120", 16384, 5120),
        # one token through an 8B-class block: the weights are read once
        _gated("gated_1x14336x4096_fp8", 1, 14336, 4096, "fp8"),
        # a decode batch of 48 through a 7B-class block
        _gated("gated_48x18944x3584_pow2", 48, 18944, 3584, "pow2"),
        # a ragged piece of a prompt through a 32B-class block, kept for training
        _gated("gated_777x27648x5120_pow2_train", 777, 27648, 5120, "pow2", quant=False, train=True),
        # the prefill of 8192 tokens through an 8B-class block
        _gated("gated_8192x14336x4096_fp8", 8192, 14336, 4096, "fp8"),
        # the gradients of a small batch: few token tiles
        _gated_bwd("gated_bwd_200x18944x3584_pow2", 200, 18944, 3584, "pow2"),
        # the gradients of a training batch of 8192 tokens
        _gated_bwd("gated_bwd_8192x14336x4096_fp8", 8192, 14336, 4096, "fp8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "gated", "gated", "gated_bwd"])
    if op in ("norm", "norm_bwd"):
        fmt = rng.choice(["bf16", "fp8", "pow2"]) if op == "norm" else "bf16"
        step = 8 if fmt == "bf16" else 128   # an output in 8 bits has whole segments
        k = step * _log(rng, max(1, 128 // step), 8192 // step)
        m = min(_log(rng, 1, 16384), 16384 * 5120 // k)
        if op == "norm_bwd":
            return _norm_bwd("", m, k, rng.random() < 0.7, rng.random() < 0.8)
        m = min(m, 8192 * 4096 // k)
        return _norm("", m, k, fmt, rng.random() < 0.7, fmt != "bf16" and rng.random() < 0.3)
    fmt = rng.choice(["fp8", "pow2"])
    n, k = 128 * _log(rng, 1, 216), 128 * _log(rng, 1, 64)
    room = 8192 * 14336 * 4096
    m = _log(rng, 1, 8192)
    m = max(1, min(m, room // (n * k)))
    if op == "gated_bwd":
        return _gated_bwd("", m, n, k, fmt)
    return _gated("", m, n, k, fmt, rng.random() < 0.6, rng.random() < 0.3)


def _scale_bytes(fmt):
    return 1 if fmt == "pow2" else 4


def work(case):
    m, k, op = case["m"], case["k"], case["op"]
    if op == "norm":
        by = 2 * m * k + 2 * k + (4 * m * k if case["residual"] else 0)
        if case["fmt"] == "bf16" or case["keep_y"]:
            by += 2 * m * k
        if case["fmt"] != "bf16":
            by += m * k + _scale_bytes(case["fmt"]) * m * (k // 128)
        return {"bytes": by, "flops": 6 * m * k}
    if op == "norm_bwd":
        by = 6 * m * k + 2 * k + (2 * m * k if case["dh"] else 0) + (4 * k if case["dw"] else 0)
        return {"bytes": by, "flops": 12 * m * k}
    n, sc = case["n"], _scale_bytes(case["fmt"])
    weights = 2 * n * k + 2 * sc * (n // 128) * (k // 128)
    if op == "gated":
        by = weights + m * k + sc * m * (k // 128) + (4 * m * n if case["train"] else 0)
        by += m * n + sc * m * (n // 128) if case["quant"] else 2 * m * n
        return {"bytes": by, "flops": 4 * m * n * k}
    return {"bytes": weights + 6 * m * n + 4 * m * k + 4 * n * k, "flops": 8 * m * n * k}


# --------------------------------------------------------------------------------- inputs

def _randn(g, shape, std):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std


def _hidden(g, m, k):
    """A residual stream: unit rows with a few strong channels, as decoder layers have them."""
    strong = torch.where(torch.rand(k, generator=g, device=DEV) < 0.002, 30.0, 1.0)
    return (_randn(g, (m, k), 1.0) * strong).to(torch.bfloat16)


def _weight(g, n, k, fmt):
    """An FP8 weight: codes uint8 [n, k] and scales of 128 x 128 blocks."""
    codes = torch.empty((n, k), dtype=torch.uint8, device=DEV)
    scales = torch.empty((n // 128, k // 128), dtype=torch.uint8 if fmt == "pow2" else torch.float32, device=DEV)
    step = max(128, (1 << 26) // k // 128 * 128)
    for i in range(0, n, step):
        w = _randn(g, (min(step, n - i), k), 0.02).view(-1, 128, k // 128, 128).transpose(1, 2)
        c, s = _encode(w.reshape(w.shape[0], w.shape[1], 128 * 128), fmt)
        codes[i:i + step] = c.view(w.shape).transpose(1, 2).reshape(-1, k).view(torch.uint8)
        scales[i // 128:(i + step) // 128] = s.view(scales.dtype)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, m, k = case["op"], case["m"], case["k"]
    st = {"case": case}
    if op in ("norm", "norm_bwd"):
        st["w"] = (1.0 + _randn(g, (k,), 0.2)).to(torch.bfloat16)
        st["x"] = _hidden(g, m, k)
        if op == "norm":
            if case["residual"]:
                st["r"] = _hidden(g, m, k)
            return st
        st["dy"] = _randn(g, (m, k), 0.01).to(torch.bfloat16)
        if case["dh"]:
            st["dh"] = _randn(g, (m, k), 0.01).to(torch.bfloat16)
    else:
        n, fmt = case["n"], case["fmt"]
        st["gate"], st["up"] = _weight(g, n, k, fmt), _weight(g, n, k, fmt)
        x = _randn(g, (m, k), 1.0)
        if op == "gated":
            c, s = _encode(x.view(m, k // 128, 128), fmt)
            st["xq"], st["sx"] = c.view(m, k).view(torch.uint8), _held(s)
        else:
            st["x"] = x.to(torch.bfloat16)
            st["gu"] = _randn(g, (m, 2 * n), 0.02 * math.sqrt(k)).to(torch.bfloat16)
            st["dh"] = _randn(g, (m, n), 0.01).to(torch.bfloat16)
    if own:
        import quantized_linear_layers_block_amd as ql
        if op == "norm_bwd":
            size = ql.binding.qlinear_rms_norm_backward_workspace(m, k)
        else:
            n, pow2 = case["n"], case["fmt"] == "pow2"
            st["weights"] = [ql.FP8Weight(c, s, n, k, pow2) for c, s in (st["gate"], st["up"])]
            size = (ql.binding.qlinear_gated_forward_workspace(m, n, k) if op == "gated" else
                    ql.binding.qlinear_gated_backward_workspace(m, n, k))
        st["ws"] = torch.zeros(size, dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------------------ plain form

def _held(scales):
    """Scales as a layer takes them: float32, or the bytes of powers of two."""
    return scales.view(torch.uint8) if scales.dtype == torch.float8_e8m0fnu else scales


def _encode(v, fmt):
    """float32 segments [.., s] -> E4M3 codes of the same shape, and the scale of each segment
    (float32, or a power of two as float8_e8m0fnu)."""
    amax = v.abs().amax(-1)
    if fmt == "pow2":
        frac, e = torch.frexp(amax)   # amax = frac 2^e, frac in [1/2, 1): 448 = (7/8) 2^9
        e = torch.where(frac <= 0.875, e - 9, e - 8).clamp(-127, 127)
        e = torch.where(amax > 0, e, torch.zeros_like(e)).to(torch.int32)
        q = torch.ldexp(v, -e[..., None])
        s = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    else:
        s = amax / 448.0
        q = torch.where(s[..., None] > 0, v / s[..., None], torch.zeros_like(v))
    return q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), s


def _scales32(s):
    return s.view(torch.float8_e8m0fnu).to(torch.float32) if s.dtype == torch.uint8 else s


def _weight32(w):
    codes, scales = w
    n, k = codes.shape
    v = codes.view(torch.float8_e4m3fn).to(torch.float32).view(n // 128, 128, k // 128, 128)
    return (v * _scales32(scales)[:, None, :, None]).view(n, k)


def _out8(v, fmt):
    m, k = v.shape
    c, s = _encode(v.view(m, k // 128, 128), fmt)
    return {"codes": c.view(m, k), "scales": s}


def _plain_norm(st):
    c = st["case"]
    x = st["x"]
    out = {}
    if c["residual"]:
        x = (x.to(torch.float32) + st["r"].to(torch.float32)).to(torch.bfloat16)
        out["h"] = x
    h = x.to(torch.float32)
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * st["w"].to(torch.float32)
    if c["fmt"] != "bf16":
        out.update(_out8(y, c["fmt"]))
    if c["fmt"] == "bf16" or c["keep_y"]:
        out["y"] = y.to(torch.bfloat16)
    return out


def _plain_norm_bwd(st):
    h, dy, w = (st[i].to(torch.float32) for i in ("x", "dy", "w"))
    s = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    a = dy * w
    dx = s * (a - h * (s * s * (a * h).mean(-1, keepdim=True)))
    if "dh" in st:
        dx = dx + st["dh"].to(torch.float32)
    out = {"dx": dx.to(torch.bfloat16)}
    if st["case"]["dw"]:
        out["dw"] = (dy * h * s).sum(0)
    return out


def _plain_gated(st):
    c = st["case"]
    m, k = st["xq"].shape
    x = st["xq"].view(torch.float8_e4m3fn).to(torch.float32).view(m, k // 128, 128)
    x = (x * _scales32(st["sx"])[..., None]).view(m, k)
    g = torch.matmul(x, _weight32(st["gate"]).t())
    u = torch.matmul(x, _weight32(st["up"]).t())
    h = g / (1.0 + torch.exp(-g)) * u
    out = _out8(h, c["fmt"]) if c["quant"] else {"h": h.to(torch.bfloat16)}
    if c["train"]:
        out["gu"] = torch.cat((g, u), 1).to(torch.bfloat16)
    return out


def _plain_gated_bwd(st):
    n = st["case"]["n"]
    g, u = st["gu"][:, :n].to(torch.float32), st["gu"][:, n:].to(torch.float32)
    dh, x = st["dh"].to(torch.float32), st["x"].to(torch.float32)
    s = 1.0 / (1.0 + torch.exp(-g))
    dg = dh * u * s * (1.0 + g * (1.0 - s))
    du = dh * g * s
    dx = torch.matmul(dg, _weight32(st["gate"])) + torch.matmul(du, _weight32(st["up"]))
    return {"dx": dx.to(torch.bfloat16), "dgate": torch.matmul(dg.t(), x).to(torch.bfloat16),
            "dup": torch.matmul(du.t(), x).to(torch.bfloat16)}


def _as_values(codes, scales):
    """Codes and scales as the types whose values they hold."""
    if scales.dtype == torch.uint8:
        scales = scales.view(torch.float8_e8m0fnu)
    return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales}


def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "gated": _plain_gated,
                "gated_bwd": _plain_gated_bwd}[op](st)
    import quantized_linear_layers_block_amd as ql
    if op == "norm":
        r = st.get("r")
        if c["fmt"] == "bf16":
            got = ql.rms_norm(st["x"], st["w"], EPS, residual=r)
            return {"y": got[0], "h": got[1]} if c["residual"] else {"y": got}
        y = torch.empty_like(st["x"]) if c["keep_y"] else None
        got = ql.rms_norm_fp8(st["x"], st["w"], EPS, residual=r, pow2=c["fmt"] == "pow2", y=y)
        out = _as_values(got[0], got[1])
        if c["residual"]:
            out["h"] = got[2]
        if c["keep_y"]:
            out["y"] = y
        return out
    if op == "norm_bwd":
        dx, dw = ql.rms_norm_backward(st["dy"], st["x"], st["w"], EPS, dh=st.get("dh"), need_dweight=c["dw"],
                                      ws=st["ws"])
        return {"dx": dx, "dw": dw} if c["dw"] else {"dx": dx}
    gate, up = st["weights"]
    if op == "gated_bwd":
        dx, dgate, dup = ql.gated_backward(gate, up, st["dh"], st["gu"], st["x"], ws=st["ws"])
        return {"dx": dx, "dgate": dgate, "dup": dup}
    gu = torch.empty((c["m"], 2 * c["n"]), dtype=torch.bfloat16, device=DEV) if c["train"] else None
    if c["quant"]:
        out = _as_values(*ql.gated_forward_fp8(gate, up, st["xq"], st["sx"], gu=gu, ws=st["ws"]))
    else:
        out = {"h": ql.gated_forward(gate, up, st["xq"], st["sx"], gu=gu, ws=st["ws"])}
    if c["train"]:
        out["gu"] = gu
    return out


# ------------------------------------------------------------------- definition, in 64 bits

def _value8(codes):
    """The float64 values of E4M3 bytes, from the fields of the format."""
    b = torch.arange(256, device=codes.device)
    e, f = (b >> 3) & 15, (b & 7).to(torch.float64)
    mag = torch.where(e == 0, f / 512.0, (1.0 + f / 8.0) * 2.0 ** (e - 7).to(torch.float64))
    return torch.where(b >= 128, -mag, mag)[codes.to(torch.int64)]


def _scale64(s):
    return 2.0 ** (s.to(torch.float64) - 127.0) if s.dtype == torch.uint8 else s.to(torch.float64)


def _weight64(w):
    codes, scales = w
    return _value8(codes) * _scale64(scales).repeat_interleave(128, 0).repeat_interleave(128, 1)


def _round8(v):
    """Nearest E4M3 value of float64 values within 448, ties to the even code."""
    a = v.abs()
    step = 2.0 ** (torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3.0)
    # log2 may round up to the next whole number just below it: the step of the value itself then
    step = torch.where(a < 8.0 * step, step / 2.0, step).clamp(min=2.0 ** -9)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), v)


def _out64(y, fmt):
    m, k = y.shape
    seg = y.view(m, k // 128, 128)
    s = seg.abs().amax(2) / 448.0
    if fmt == "pow2":
        e = torch.ceil(torch.log2(s.clamp(min=2.0 ** -127)))
        e = torch.where(s <= 2.0 ** (e - 1.0), e - 1.0, torch.where(s > 2.0 ** e, e + 1.0, e)).clamp(-127, 127)
        s = torch.where(s > 0, 2.0 ** e, torch.ones_like(s))
    q = torch.where(s[..., None] > 0, seg / s.clamp(min=1e-300)[..., None], torch.zeros_like(seg))
    return {"codes": _round8(q).view(m, k), "scales": s}


def exact(case, seed):
    st = prepare(case, seed)
    op, m, k = case["op"], case["m"], case["k"]
    if op == "norm":
        out = {}
        h = st["x"].to(torch.float64)
        if case["residual"]:
            # the residual stream is held in bf16, and the norm is the norm of what is held
            h = (h + st["r"].to(torch.float64)).to(torch.bfloat16).to(torch.float64)
            out["h"] = h
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / k + EPS) * st["w"].to(torch.float64)
        if case["fmt"] != "bf16":
            out.update(_out64(y, case["fmt"]))
        if case["fmt"] == "bf16" or case["keep_y"]:
            out["y"] = y
        return out
    if op == "norm_bwd":
        h, dy, w = (st[i].to(torch.float64) for i in ("x", "dy", "w"))
        z = torch.sqrt(h.square().sum(1, keepdim=True) / k + EPS)
        a = dy * w
        dx = a / z - h * (a * h).sum(1, keepdim=True) / (k * z ** 3)
        if case["dh"]:
            dx += st["dh"].to(torch.float64)
        return {"dx": dx, "dw": torch.mv((dy * h).t(), 1.0 / z[:, 0])} if case["dw"] else {"dx": dx}
    n = case["n"]
    if op == "gated":
        x = _value8(st["xq"]) * _scale64(st["sx"]).repeat_interleave(128, 1)
        g = torch.mm(x, _weight64(st["gate"]).t().contiguous())
        u = torch.mm(x, _weight64(st["up"]).t().contiguous())
        h = g * torch.sigmoid(g) * u
        out = _out64(h, case["fmt"]) if case["quant"] else {"h": h}
        if case["train"]:
            out["gu"] = torch.cat((g, u), 1)
        return out
    g, u = st["gu"][:, :n].to(torch.float64), st["gu"][:, n:].to(torch.float64)
    dh, x = st["dh"].to(torch.float64), st["x"].to(torch.float64)
    s = torch.sigmoid(g)
    dg, du = dh * u * (s + g * s * (1.0 - s)), dh * g * s
    dx = torch.mm(dg, _weight64(st["gate"]))
    dx += torch.mm(du, _weight64(st["up"]))
    return {"dx": dx, "dgate": torch.mm(dg.t().contiguous(), x), "dup": torch.mm(du.t().contiguous(), x)}
