"""MI355X (gfx950) quantized rollout linear layer: NVFP4 and blockwise-FP8 weights with a bf16
LoRA adapter, behind the C ABI of include/qlinear.h.

    y = x . dequant(Wq)^T + s . (x A^T) B^T

``binding`` is the one-to-one ctypes binding of the C entry points (same names).  The
helpers below only allocate the output and workspace tensors with PyTorch (device memory
and the current stream are all PyTorch is used for) and call the binding; every step of
the layer runs in the HIP kernels of libqlinear.so.  Importing the package fails if the
library has not been built -- there is no fallback.
"""
from dataclasses import dataclass

import torch

from . import binding
from .binding import (QL_FP8_BLOCK128, QL_FP8_POW2, QL_NVFP4, QL_OUT_BF16, QL_OUT_F32,  # noqa: F401
                      QlinearError, make_qweight)

__all__ = ["NVFP4Weight", "FP8Weight", "quantize_nvfp4", "quantize_fp8_block", "quantize_act_fp8",
           "forward", "forward_fp8_prequant", "RequantTable", "QlinearError", "binding", "workspace_status",
           "quantize_fp8_pow2", "kv_store_fp8", "kv_load_fp8", "KVCacheNVFP4", "kv_store_nvfp4", "kv_load_nvfp4",
           "attention_nvfp4", "rms_norm", "rms_norm_fp8", "rms_norm_backward",
           "gated_forward", "gated_forward_fp8", "gated_backward"]


def _dev(t):
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    return t


@dataclass
class NVFP4Weight:
    codes: torch.Tensor         # uint8 [n, k/2]
    scales: torch.Tensor        # uint8 [n, k/16] (E4M3)
    tensor_scale: torch.Tensor  # float32 [1]
    n: int
    k: int

    def qweight(self):
        return make_qweight(QL_NVFP4, self.n, self.k, self.codes, self.scales, self.tensor_scale)

    @staticmethod
    def empty(n, k, device="cuda"):
        return NVFP4Weight(torch.empty((n, k // 2), dtype=torch.uint8, device=device),
                           torch.empty((n, k // 16), dtype=torch.uint8, device=device),
                           torch.empty((1,), dtype=torch.float32, device=device), n, k)


@dataclass
class FP8Weight:
    codes: torch.Tensor   # uint8 [n, k] (E4M3)
    scales: torch.Tensor  # float32 [n/128, k/128], or uint8 E8M0 bytes with pow2
    n: int
    k: int
    pow2: bool = False    # power-of-two block scales (QL_FP8_POW2)

    def qweight(self):
        return make_qweight(QL_FP8_POW2 if self.pow2 else QL_FP8_BLOCK128, self.n, self.k, self.codes,
                            self.scales, None)

    @staticmethod
    def empty(n, k, device="cuda", pow2=False):
        return FP8Weight(torch.empty((n, k), dtype=torch.uint8, device=device),
                         torch.empty((n // 128, k // 128), dtype=torch.uint8 if pow2 else torch.float32,
                                     device=device), n, k, pow2)


def _u16(t):
    if t.dtype != torch.bfloat16:
        raise TypeError("bf16 tensors expected")
    return t


def _ws(nbytes, device):
    # zero-filled: a workspace starts with the status word and the workgroup counters
    return torch.zeros((max(int(nbytes), 1),), dtype=torch.uint8, device=device)


def workspace_status(ws):
    """Status word (QLINEAR_STATUS_* bits) of a forward or requantization workspace."""
    return int(ws[:4].view(torch.int32).item())


def quantize_nvfp4(w, out=None, status_word=None):
    _dev(_u16(w))
    n, k = w.shape
    q = out if out is not None else NVFP4Weight.empty(n, k, w.device)
    ws = _ws(binding.qlinear_quantize_workspace(QL_NVFP4, n, k), w.device)
    binding.qlinear_quantize_nvfp4(w, q.codes, q.scales, q.tensor_scale, ws, status_word)
    return q


def quantize_fp8_block(w, out=None, status_word=None):
    _dev(_u16(w))
    n, k = w.shape
    q = out if out is not None else FP8Weight.empty(n, k, w.device)
    binding.qlinear_quantize_fp8_block(w, q.codes, q.scales, status_word)
    return q


def quantize_fp8_pow2(w, out=None, status_word=None):
    _dev(_u16(w))
    n, k = w.shape
    q = out if out is not None else FP8Weight.empty(n, k, w.device, pow2=True)
    binding.qlinear_quantize_fp8_pow2(w, q.codes, q.scales, status_word)
    return q


def quantize_act_fp8(x, pow2=False):
    _dev(_u16(x))
    m, k = x.shape
    xq = torch.empty((m, k), dtype=torch.uint8, device=x.device)
    sx = torch.empty((m, k // 128), dtype=torch.uint8 if pow2 else torch.float32, device=x.device)
    (binding.qlinear_quantize_act_fp8_pow2 if pow2 else binding.qlinear_quantize_act_fp8)(x, xq, sx)
    return xq, sx


def _fmt(qw):
    if isinstance(qw, NVFP4Weight):
        return QL_NVFP4
    return QL_FP8_POW2 if qw.pow2 else QL_FP8_BLOCK128


def forward(qw, x, lora_a=None, lora_b=None, lora_scale=0.0, out_dtype=torch.bfloat16, out=None, ws=None):
    """y = x . dequant(qw)^T + lora_scale (x A^T) B^T  (bf16 or float32 output)."""
    _dev(_u16(x))
    m = x.shape[0]
    rank = 0 if lora_a is None else lora_a.shape[0]
    if out is None:
        out = torch.empty((m, qw.n), dtype=out_dtype, device=x.device)
    od = QL_OUT_F32 if out.dtype == torch.float32 else QL_OUT_BF16
    eff_rank = rank if (lora_a is not None and lora_b is not None and lora_scale != 0) else 0
    if ws is None:
        ws = _ws(binding.qlinear_forward_workspace(_fmt(qw), m, qw.n, qw.k, eff_rank), x.device)
    binding.qlinear_forward(qw.qweight(), x, out, od, ws, lora_a, lora_b, rank, lora_scale)
    return out


def forward_group(qws, x, loras=None, lora_scale=0.0, out_dtype=torch.bfloat16, outs=None, ws=None):
    """Several NVFP4 layers on the same x (a fused q/k/v or gate/up projection): returns
    [x . dequant(qw)^T + lora_scale (x A^T) B^T for each qw]; loras is a list of (A, B)."""
    _dev(_u16(x))
    m = x.shape[0]
    if loras is None:
        loras = [(None, None)] * len(qws)
    rank = 0 if loras[0][0] is None else loras[0][0].shape[0]
    if outs is None:
        outs = [torch.empty((m, qw.n), dtype=out_dtype, device=x.device) for qw in qws]
    od = QL_OUT_F32 if outs[0].dtype == torch.float32 else QL_OUT_BF16
    with_lora = all(a is not None and b is not None for a, b in loras)
    eff_rank = rank if (with_lora and lora_scale != 0) else 0
    if ws is None:
        ws = _ws(binding.qlinear_forward_group_workspace(m, qws[0].k, [qw.n for qw in qws], eff_rank), x.device)
    layers = [(qw.qweight(), a, b, y) for qw, (a, b), y in zip(qws, loras, outs)]
    binding.qlinear_forward_group(layers, x, od, ws, rank, lora_scale)
    return outs


def forward_fp8_prequant(qw, xq, sx, x=None, lora_a=None, lora_b=None, lora_scale=0.0,
                         out_dtype=torch.bfloat16, out=None, ws=None):
    m = xq.shape[0]
    rank = 0 if lora_a is None else lora_a.shape[0]
    if out is None:
        out = torch.empty((m, qw.n), dtype=out_dtype, device=xq.device)
    od = QL_OUT_F32 if out.dtype == torch.float32 else QL_OUT_BF16
    eff_rank = rank if (lora_a is not None and lora_b is not None and lora_scale != 0) else 0
    if ws is None:
        ws = _ws(binding.qlinear_forward_prequant_workspace(m, qw.n, qw.k, eff_rank), xq.device)
    binding.qlinear_forward_fp8_prequant(qw.qweight(), xq, sx, out, od, ws, x, lora_a, lora_b, rank, lora_scale)
    return out


def backward(qw, dy, x=None, lora_a=None, lora_b=None, lora_scale=0.0, dx_dtype=torch.bfloat16, ws=None):
    """Gradients of the NVFP4 layer with LoRA: (dx, da, db); da, db are float32 (None
    without an adapter)."""
    _dev(_u16(dy))
    if not isinstance(qw, NVFP4Weight):
        raise TypeError("the backward pass is defined for NVFP4 weights")
    m = dy.shape[0]
    rank = 0 if lora_a is None else lora_a.shape[0]
    eff_rank = rank if (lora_a is not None and lora_b is not None and lora_scale != 0) else 0
    dx = torch.empty((m, qw.k), dtype=dx_dtype, device=dy.device)
    da = torch.empty((rank, qw.k), dtype=torch.float32, device=dy.device) if eff_rank else None
    db = torch.empty((qw.n, rank), dtype=torch.float32, device=dy.device) if eff_rank else None
    if ws is None:
        nb = binding.qlinear_backward_workspace(QL_NVFP4, m, qw.n, qw.k, eff_rank)
        ws = _ws(nb, dy.device) if nb else None
    od = QL_OUT_F32 if dx_dtype == torch.float32 else QL_OUT_BF16
    binding.qlinear_backward(qw.qweight(), x, dy, dx, od, da, db, ws, lora_a, lora_b, rank, lora_scale)
    return dx, da, db


class RequantTable:
    """A whole policy to requantize after every training step: a list of (bf16 weight,
    quantized weight) pairs, whose item array is copied to the device once."""

    def __init__(self, pairs, fmt=QL_NVFP4, device="cuda"):
        self.pairs = list(pairs)   # keep the tensors alive
        self.fmt = fmt
        img = binding.requant_items_bytes([(w, q.qweight()) for w, q in self.pairs])
        self.items = torch.frombuffer(bytearray(img), dtype=torch.uint8).to(device)
        self.ws = _ws(binding.qlinear_requant_workspace(len(self.pairs)), device)

    def requantize_all(self):
        binding.qlinear_requantize_all(self.items, len(self.pairs), self.fmt, self.ws)

    def set_updates(self, deltas):
        """Device pointer array of one dense bf16 update per tensor (kept alive here)."""
        self.deltas = list(deltas)
        ptrs = torch.tensor([d.data_ptr() for d in self.deltas], dtype=torch.int64)
        self.delta_ptrs = ptrs.to(self.ws.device)

    def update_requantize_all(self):
        """W <- bf16(W + delta) for every tensor, fused with the requantization."""
        binding.qlinear_update_requantize_all(self.items, self.delta_ptrs, len(self.pairs), self.fmt, self.ws)

    def status(self):
        """The workspace's status word (QLINEAR_STATUS_* bits); synchronises."""
        return int(self.ws[:4].view(torch.int32).item())


def kv_store_fp8(kv, slots, cache_codes, cache_scales, status_word=None):
    """Store bf16 kv [T, H, D] into FP8 cache rows slots[t] (codes u8 [S, H, D], scales f32 [S, H])."""
    binding.qlinear_kv_store_fp8(_dev(_u16(kv)), slots, cache_codes, cache_scales, status_word)


def kv_load_fp8(cache_codes, cache_scales, slots, heads=None, status_word=None):
    """Load cache rows `slots` back to bf16 [T, H, D]."""
    t = slots.shape[0]
    out = torch.empty((t, cache_codes.shape[1], cache_codes.shape[2]), dtype=torch.bfloat16,
                      device=cache_codes.device)
    binding.qlinear_kv_load_fp8(cache_codes, cache_scales, slots, out, status_word)
    return out


@dataclass(frozen=True, eq=False)
class KVCacheNVFP4:
    """A paged KV cache in 4 bits: data uint8 [pages, heads, page_size / 16, 18 D + 32] (the
    layout is in include/qlinear.h).  Slot s is token s % page_size of page s // page_size."""
    data: torch.Tensor
    pages: int
    heads: int
    head_dim: int
    page_size: int

    def __post_init__(self):
        d = self.data
        need = binding.qlinear_kv_nvfp4_bytes(self.pages, self.page_size, self.heads, self.head_dim)
        if need == 0:
            raise ValueError("page_size is a power of two in [16, 1024], head_dim 64, 128 or 256")
        if d.dtype != torch.uint8 or not d.is_contiguous() or d.numel() != need:
            raise ValueError(f"data must be {need} contiguous bytes")
        # (frozen: the handle holds the address of data)
        object.__setattr__(self, "handle", binding.make_kv_nvfp4(d, self.pages, self.page_size, self.heads, self.head_dim))
        object.__setattr__(self, "device", d.device)

    @staticmethod
    def empty(pages, heads, head_dim, page_size=64, device="cuda"):
        """A cache of pages * page_size slots; what was never stored may hold anything."""
        data = torch.empty((pages, heads, page_size // 16, 18 * head_dim + 32), dtype=torch.uint8, device=device)
        return KVCacheNVFP4(data, pages, heads, head_dim, page_size)


# Checks of the cache's calls.  A decode step makes several of them a layer, so they are few
# attribute reads each; the messages are put together only when one fails.
_BF16, _I32 = torch.bfloat16, torch.int32
_device_now = None   # (looked up by the first call on the GPU; a PyTorch for hosts alone has none)


def _refuse(device, dtype, name, t, what):
    if t.device != device:
        raise ValueError(f"{name} must live on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    raise ValueError(f"{name} must be {what}")


def _cache_device(cache):
    dev = cache.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on the GPU")
    return dev


def _check_rows(device, name, t, shape):
    # the rows of a token are dense; tokens may be apart (part of a fused projection)
    if t.shape != shape or t.dtype is not _BF16 or t.device != device:
        _refuse(device, _BF16, name, t, f"of the shape {tuple(shape)}")
    if not t.is_contiguous() and shape[0]:
        st = t.stride()
        if st[2] != 1 or (shape[1] > 1 and st[1] != shape[2]):
            raise ValueError(f"{name} must have dense [heads, head_dim] rows")


def _check_dense(device, dtype, name, t, shape):
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        _refuse(device, dtype, name, t, f"a contiguous tensor of the shape {tuple(shape)}")


def _call_on(device, fn, *args):
    """fn(*args) with `device` current, on its current stream."""
    global _device_now
    if _device_now is None:
        _device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    if _device_now() == device.index:
        return fn(*args)
    with torch.cuda.device(device):
        return fn(*args)


def kv_store_nvfp4(k, v, slots, cache, status_word=None):
    """Store bf16 keys and values [T, H, D] in slots[t] (int64, distinct) of an NVFP4 cache."""
    dev = _cache_device(cache)
    t = slots.numel()
    shape = (t, cache.heads, cache.head_dim)
    _check_rows(dev, "k", k, shape)
    _check_rows(dev, "v", v, shape)
    _check_dense(dev, torch.int64, "slots", slots, (t,))
    if status_word is not None:
        _check_dense(dev, _I32, "status_word", status_word, (1,))
    if t:
        _call_on(dev, binding.qlinear_kv_store_nvfp4, cache.handle, k, v, slots, status_word)


def kv_load_nvfp4(cache, slots, k_out=None, v_out=None, status_word=None):
    """(k, v) bf16 [T, H, D] of the cache's slots[t]."""
    dev = _cache_device(cache)
    t = slots.numel()
    shape = (t, cache.heads, cache.head_dim)
    _check_dense(dev, torch.int64, "slots", slots, (t,))
    if status_word is not None:
        _check_dense(dev, _I32, "status_word", status_word, (1,))
    if k_out is None:
        k_out = torch.empty(shape, dtype=_BF16, device=dev)
    else:
        _check_rows(dev, "k_out", k_out, shape)
    if v_out is None:
        v_out = torch.empty_like(k_out) if k_out.is_contiguous() else torch.empty(shape, dtype=_BF16, device=dev)
    else:
        _check_rows(dev, "v_out", v_out, shape)
    if t:
        _call_on(dev, binding.qlinear_kv_load_nvfp4, cache.handle, slots, k_out, v_out, status_word)
    return k_out, v_out


def attention_nvfp4(q, cache, page_table, kv_lens, q_starts=None, max_q_len=None, softmax_scale=None, causal=True,
                    window=0, out=None, lse=None, ws=None):
    """Attention of bf16 queries [Tq, Hq, D] over an NVFP4 cache: out bf16 [Tq, Hq, D].

    page_table int32 [B, P] and kv_lens int32 [B] name each sequence's cached tokens, those of
    its own queries included.  Without q_starts every sequence has Tq / B query tokens; with it
    (int32 [B + 1]) sequence b has tokens [q_starts[b], q_starts[b + 1]), at most max_q_len.
    softmax_scale defaults to 1 / sqrt(D).  causal aligns the last query with the last cached
    token; window > 0 keeps the last `window` tokens.  lse (float32 [Tq, Hq]) is filled if
    given.  ws: a zero-filled workspace kept from call to call, as forward's; without one the
    call makes its own, and with it goes the status word that tells of pages, lengths and
    q_starts outside their bounds (the call leaves them out).  No query tokens: an empty
    result, nothing is launched.  out may be q itself."""
    dev = _cache_device(cache)
    if q.dim() != 3 or q.shape[2] != cache.head_dim:
        raise ValueError(f"q must be [tokens, heads, {cache.head_dim}]")
    shape = q.shape
    tq, hq, d = shape
    if q.dtype is not _BF16 or q.device != dev or not q.is_contiguous():
        _check_rows(dev, "q", q, shape)
    batch = kv_lens.shape[0]
    _check_dense(dev, _I32, "kv_lens", kv_lens, (batch,))
    if page_table.dtype is not _I32 or page_table.dim() != 2 or page_table.shape[0] != batch or \
            page_table.device != dev or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        _refuse(dev, _I32, "page_table", page_table, "[batch, pages] with dense rows")
    if q_starts is not None:
        _check_dense(dev, _I32, "q_starts", q_starts, (batch + 1,))
        if max_q_len is None:
            raise ValueError("q_starts needs max_q_len")
    elif max_q_len is None:
        max_q_len = tq // max(batch, 1)
    if not (-0x80000000 <= max_q_len <= 0x7FFFFFFF and -0x80000000 <= window <= 0x7FFFFFFF):
        raise ValueError("max_q_len and window are 32-bit numbers")
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else torch.empty(shape, dtype=_BF16, device=dev)
    else:
        _check_rows(dev, "out", out, shape)
    if lse is not None:
        _check_dense(dev, torch.float32, "lse", lse, (tq, hq))
    if tq == 0:
        if hq == 0 or hq % cache.heads:
            raise ValueError(f"q must have a multiple of {cache.heads} heads")
        return out
    if ws is None:
        ws = _ws(binding.qlinear_attention_nvfp4_workspace(batch, tq, hq, cache.heads, d, max_q_len), dev)
    elif ws.device != dev or not ws.is_contiguous():
        _refuse(dev, ws.dtype, "ws", ws, "contiguous")
    _call_on(dev, binding.qlinear_attention_nvfp4, cache.handle, q, page_table, kv_lens, out, ws, q_starts, max_q_len,
             d ** -0.5 if softmax_scale is None else softmax_scale, causal, window, lse)
    return out


# ------------------------------------------------------------------------ norm

_U8, _F32 = torch.uint8, torch.float32


def _check_matrix(device, name, t, shape):
    # the row stride of a matrix of dense rows, which may be apart
    if t.shape != shape or t.dtype is not _BF16 or t.device != device:
        _refuse(device, _BF16, name, t, f"of the shape {tuple(shape)}")
    if t.is_contiguous():
        return shape[1]
    if shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have dense rows")
    return t.stride(0) if shape[0] > 1 else shape[1]


def _norm_device(name, t):
    dev = t.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on the GPU")
    if t.dim() != 2:
        raise ValueError(f"{name} must be [tokens, k]")
    return dev


def _norm(x, weight, eps, residual, h, y, fmt, pow2):
    # both forms of the norm: (y or None, yq, sy, h)
    dev = _norm_device("x", x)
    shape = x.shape
    k = shape[1]
    xs = _check_matrix(dev, "x", x, shape)
    if weight.shape != (k,) or weight.dtype is not _BF16 or weight.device != dev or not weight.is_contiguous():
        _check_dense(dev, _BF16, "weight", weight, (k,))
    rs = hs = 0
    if residual is not None:
        rs = _check_matrix(dev, "residual", residual, shape)
        if h is None:
            h, hs = torch.empty_like(x) if xs == k else torch.empty(shape, dtype=_BF16, device=dev), k
    if h is not None and not hs:
        hs = _check_matrix(dev, "h", h, shape)
    yq = sy = None
    if fmt:
        if y is not None:
            _check_dense(dev, _BF16, "y", y, shape)
        yq = torch.empty(shape, dtype=_U8, device=dev)
        sy = torch.empty((shape[0], k // 128), dtype=_U8 if pow2 else _F32, device=dev)
    elif y is not None:
        _check_dense(dev, _BF16, "out", y, shape)
    else:
        y = torch.empty_like(x) if xs == k else torch.empty(shape, dtype=_BF16, device=dev)
    _call_on(dev, binding.qlinear_rms_norm, x, xs, weight, eps, residual, rs, h, hs, y, fmt, yq, sy)
    return y, yq, sy, h


def rms_norm(x, weight, eps=1e-6, residual=None, h=None, out=None):
    """y = h / sqrt(mean(h^2) + eps) * weight of bf16 rows [T, k], h = bf16(x + residual): y, or
    (y, h) with a residual.  h (given, it is written also without one) may be x or residual itself;
    y is written into out if given."""
    y, _, _, h = _norm(x, weight, eps, residual, h, out, 0, False)
    return y if residual is None else (y, h)


def rms_norm_fp8(x, weight, eps=1e-6, residual=None, pow2=False, h=None, y=None):
    """rms_norm with an output in 8 bits for the FP8 layers: (yq, sy), or (yq, sy, h) with a
    residual; yq uint8 [T, k] E4M3 codes, sy float32 [T, k / 128] (pow2: uint8 E8M0 bytes).  y
    (bf16 [T, k]), if given, is written too, for an adapter or a weight gradient."""
    _, yq, sy, h = _norm(x, weight, eps, residual, h, y, QL_FP8_POW2 if pow2 else QL_FP8_BLOCK128, pow2)
    return (yq, sy) if residual is None else (yq, sy, h)


def rms_norm_backward(dy, h, weight, eps=1e-6, dh=None, dx=None, need_dweight=True, ws=None):
    """Gradients of rms_norm: (dx, dweight).  dy is the gradient of y, h what the forward
    normalised, dh the gradient that reaches h beside the norm (added to dx).  dx (bf16; dy or dh
    itself if wanted) is the gradient of x and of the residual; dweight is float32 [k], None
    without need_dweight.  ws: scratch kept from step to step."""
    dev = _norm_device("dy", dy)
    shape = dy.shape
    m, k = shape
    ds = _check_matrix(dev, "dy", dy, shape)
    hs = _check_matrix(dev, "h", h, shape)
    _check_dense(dev, _BF16, "weight", weight, (k,))
    dhs = 0 if dh is None else _check_matrix(dev, "dh", dh, shape)
    if dx is None:
        dx, dxs = torch.empty_like(dy) if ds == k else torch.empty(shape, dtype=_BF16, device=dev), k
    else:
        dxs = _check_matrix(dev, "dx", dx, shape)
    dweight = None
    if need_dweight:
        dweight = torch.empty((k,), dtype=_F32, device=dev)
        if ws is None:
            ws = torch.empty((max(1, binding.qlinear_rms_norm_backward_workspace(m, k)),), dtype=_U8, device=dev)
        elif ws.device != dev or not ws.is_contiguous():
            _refuse(dev, ws.dtype, "ws", ws, "contiguous")
    _call_on(dev, binding.qlinear_rms_norm_backward, dy, ds, h, hs, weight, eps, dx, dxs, dh, dhs, dweight,
             ws if need_dweight else None)
    return dx, dweight


# --------------------------------------------------- gated feed-forward block

def _gated_weights(gate, up):
    # the device of a block's weights
    if not isinstance(gate, FP8Weight) or not isinstance(up, FP8Weight):
        raise TypeError("the gated block takes FP8 weights")
    n, k, pow2 = gate.n, gate.k, gate.pow2
    if n != up.n or k != up.k or pow2 != up.pow2:
        raise ValueError("gate and up must be alike in sizes and scales")
    dev = gate.codes.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on the GPU")
    codes, scales, kind = (n, k), (n // 128, k // 128), _U8 if pow2 else _F32
    for w in (gate, up):
        _check_dense(dev, _U8, "codes", w.codes, codes)
        _check_dense(dev, kind, "scales", w.scales, scales)
    return dev


def _gated_call(gate, up, xq, sx, h, gu, ws, quant):
    # both forms of the forward: (h, hq, sh)
    dev = _gated_weights(gate, up)
    if xq.dim() != 2:
        raise ValueError("xq must be [tokens, k]")
    m, n, k = xq.shape[0], gate.n, gate.k
    _check_dense(dev, _U8, "xq", xq, (m, k))
    _check_dense(dev, gate.scales.dtype, "sx", sx, (m, k // 128))
    if h is not None:
        _check_dense(dev, _BF16, "h", h, (m, n))
    if gu is not None:
        _check_dense(dev, _BF16, "gu", gu, (m, 2 * n))
    if ws is None:
        ws = _ws(binding.qlinear_gated_forward_workspace(m, n, k), dev)
    elif ws.device != dev or not ws.is_contiguous():
        _refuse(dev, ws.dtype, "ws", ws, "contiguous")
    hq = sh = None
    if quant:
        hq, sh = xq.new_empty((m, n)), sx.new_empty((m, n // 128))
    elif h is None:
        h = torch.empty((m, n), dtype=_BF16, device=dev)
    _call_on(dev, binding.qlinear_gated_forward, gate.qweight(), up.qweight(), xq, sx, ws, h, hq, sh, gu)
    return h, hq, sh


def gated_forward(gate, up, xq, sx, h=None, gu=None, ws=None):
    """h = silu(x Wg^T) * (x Wu^T), bf16 [T, n], from FP8 weights and activations quantized like them
    (rms_norm_fp8, quantize_act_fp8).  gu (bf16 [T, 2n]), if given, gets both products, for
    gated_backward.  With pow2 weights the sums drop what is 13 bits below the largest of eight
    products (1.4e-5 of g on normal data).  ws: a zero-filled workspace kept from call to call, as
    forward's."""
    return _gated_call(gate, up, xq, sx, h, gu, ws, False)[0]


def gated_forward_fp8(gate, up, xq, sx, h=None, gu=None, ws=None):
    """gated_forward with an output in 8 bits for the down projection's forward_fp8_prequant:
    (hq uint8 [T, n], sh [T, n / 128]); h (bf16 [T, n]), if given, is written too."""
    return _gated_call(gate, up, xq, sx, h, gu, ws, True)[1:]


def gated_backward(gate, up, dh, gu, x=None, need_dx=True, need_dweight=True, ws=None):
    """Gradients of gated_forward: (dx, dgate, dup), bf16 [T, k] and [n, k] twice (None where not
    wanted).  dh (bf16 [T, n]) is the gradient of h, gu what the forward filled, x (bf16 [T, k]) the
    activations before their quantization, needed for the weights' gradients.  ws: scratch kept
    from step to step."""
    dev = _gated_weights(gate, up)
    n, k = gate.n, gate.k
    if dh.dim() != 2:
        raise ValueError("dh must be [tokens, n]")
    m = dh.shape[0]
    _check_dense(dev, _BF16, "dh", dh, (m, n))
    _check_dense(dev, _BF16, "gu", gu, (m, 2 * n))
    dx = dgate = dup = None
    if need_dweight:
        if x is None:
            raise ValueError("the weights' gradients need x")
        _check_dense(dev, _BF16, "x", x, (m, k))
        dgate = torch.empty((n, k), dtype=_BF16, device=dev)
        dup = torch.empty((n, k), dtype=_BF16, device=dev)
    if need_dx:
        dx = torch.empty((m, k), dtype=_BF16, device=dev)
    if ws is None:
        ws = torch.empty((max(1, binding.qlinear_gated_backward_workspace(m, n, k)),), dtype=_U8, device=dev)
    elif ws.device != dev or not ws.is_contiguous():
        _refuse(dev, ws.dtype, "ws", ws, "contiguous")
    _call_on(dev, binding.qlinear_gated_backward, gate.qweight(), up.qweight(), dh, gu, ws, x, dx, dgate, dup)
    return dx, dgate, dup
