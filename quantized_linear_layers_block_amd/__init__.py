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
           "attention_nvfp4"]


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
