"""The operators of the 4-bit KV cache, as cases to measure: storing keys and values in NVFP4
rows, loading them back, and attention that reads the cache.

A cache is one uint8 tensor [pages][heads][page_size / 16][18 D + 32]: groups of 16 tokens of
one head.  A group holds
    K codes  [16 t][D/2]                two E2M1 codes a byte, the even element in the low nibble
    K scales [16 t][D/16]               E4M3, one for 16 elements
    K exps   [16 t]                     e + 127 of the row's scale 2^e
    V codes  [4 t/4][16 m][D/32 j][4 t%4]   the byte of elements 2p and 2p + 1, p = 16 j + m
    V scales [4 t/4][2 b%2][D/32 b/2][4 t%4]  E4M3 of the block b of 16 elements
    V exps   [16 t]
and an element is E2M1(code) * E4M3(scale) * 2^e.  Slot s of the cache is token s % page_size
of page s / page_size; a sequence's tokens are found through its row of the page table.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------- cases

def _att(name, batch, ctx, q_heads, kv_heads, head_dim, page, q_len=1, ragged=False, mixed=False, causal=True,
         window=0, lse=False):
    c = dict(op="attention", batch=batch, ctx=ctx, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page=page,
             q_len=q_len, ragged=ragged, mixed=mixed, causal=causal, window=window, lse=lse)
    return dict(name=name, **c) if name else c


def _copy(name, op, tokens, kv_heads, head_dim, page):
    c = dict(op=op, tokens=tokens, kv_heads=kv_heads, head_dim=head_dim, page=page)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one user's next token on a 7B-class layer (28 query and 4 KV heads): latency alone
        _att("decode_1x613_28h4", 1, 613, 28, 4, 128, 16),
        # a serving batch on a 32B-class layer (64 / 8 heads), about 3000 tokens a sequence
        _att("decode_64x4096_64h8", 64, 4096, 64, 8, 128, 64, ragged=True),
        # a rollout batch of 256 sequences of every length up to 4096
        _att("decode_256x4096_64h8", 256, 4096, 64, 8, 128, 16, ragged=True),
        # few sequences with a long memory: the work has to be split along the tokens
        _att("decode_3x131071_28h4", 3, 131071, 28, 4, 128, 128, lse=True),
        # checking 4 drafted tokens a sequence, wide heads
        _att("verify_24x5_on_3001_16h8_d256", 24, 3001, 16, 8, 256, 32, q_len=5, ragged=True),
        # a whole prompt against its own keys, just stored
        _att("prompt_1x8192_28h4", 1, 8192, 28, 4, 128, 64, q_len=8192),
        # the next pieces of four long prompts
        _att("chunk_4x512_on_16384_64h8", 4, 16384, 64, 8, 128, 64, q_len=512, ragged=True),
        # decoding sequences and prompt pieces in one batch, narrow heads, a sliding window
        _att("mixed_40x333_window_d64", 40, 5000, 32, 8, 64, 16, q_len=333, ragged=True, mixed=True, window=1024,
             lse=True),
        # the new tokens of a decode step are written and read back
        _copy("store_256_8h", "store", 256, 8, 128, 16),
        # four prompts of 4096 tokens are written and read back
        _copy("store_16384_8h", "store", 16384, 8, 128, 64),
        # a short prefix is read back for a layer that wants bf16, odd sizes
        _copy("load_777_4h_d64", "load", 777, 4, 64, 32),
        # a long shared prefix is read back
        _copy("load_65536_8h", "load", 65536, 8, 128, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    head_dim = rng.choice([64, 128, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    kind = rng.choice(["decode", "decode", "verify", "prompt", "chunk", "mixed", "store", "load"])
    if kind in ("store", "load"):
        top = 16384 if kind == "store" else 65536
        return _copy("", kind, min(_log(rng, 1, top), top * 128 // head_dim), rng.choice([1, 2, 4, 8]), head_dim, page)
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    batch = _log(rng, 1, 256)
    lse = rng.random() < 0.3
    room = 600_000_000 // (kv_heads * (18 * head_dim + 32) // 16)  # tokens of the whole cache
    if kind in ("decode", "verify"):
        q_len = 1 if kind == "decode" else rng.randint(2, 8)
        top = max(64, min(131072, room // batch))
        ctx = max(q_len, _log(rng, 8, top))
        window = rng.choice([0, 0, 0, rng.randint(1, 2048)])
        return _att("", batch, ctx, kv_heads * group, kv_heads, head_dim, page, q_len, rng.random() < 0.7, False,
                    True, window, lse)
    batch = _log(rng, 1, 16)
    q_len = _log(rng, 65, 8192 if kind == "prompt" else 2048)
    ctx = q_len if kind == "prompt" else q_len + _log(rng, 16, 16384)
    q_heads = kv_heads * group
    while 4.0 * head_dim * q_heads * q_len * ctx * batch > 5e11:
        if batch > 1:
            batch = (batch + 1) // 2
        elif ctx > q_len + 64:
            ctx = (ctx + q_len) // 2
        else:
            q_len = ctx = max(65, q_len // 2)
    causal = kind != "prompt" or rng.random() < 0.7
    window = rng.randint(1, 4096) if causal and rng.random() < 0.25 else 0
    return _att("", batch, ctx, q_heads, kv_heads, head_dim, page, q_len, rng.random() < 0.5, kind == "mixed", causal,
                window, lse)


def _lens(case):
    """(query tokens, cached tokens) of each sequence; the cached ones include the queries'."""
    out = []
    for b in range(case["batch"]):
        u = ((b + 1) * 0.6180339887498949) % 1.0   # spread evenly over (0, 1)
        w = ((b + 1) * 0.7548776662466927) % 1.0
        q = case["q_len"]
        if case["mixed"]:
            q = 1 if b % 2 == 0 else max(1, int(q * w))
        n = case["ctx"]
        if case["ragged"]:
            n = max(q, int(n * (0.5 + 0.5 * u))) if case["batch"] < 128 else max(q, 1 + int((n - 1) * u))
        out.append((q, n))
    return out


def _visible(case, q, n):
    """(query, key) pairs of one sequence that attend, and the keys any query sees."""
    w = case["window"]
    if not case["causal"]:
        return q * n, n
    pairs = 0
    if not w:
        pairs = q * n - q * (q - 1) // 2
        return pairs, n
    for i in range(q):
        pairs += min(w, n - q + i + 1)
    return pairs, min(n, q + w - 1)


def work(case):
    d, h = case["head_dim"], case["kv_heads"]
    row = d // 2 + d // 16 + 1
    if case["op"] in ("store", "load"):
        t = case["tokens"]
        values = 4 * t * h * d
        if case["op"] == "store":   # read bf16, write rows; read rows, write bf16
            return {"bytes": 2 * values + 2 * 2 * t * h * row + 8 * t, "flops": 2 * t * h * d * 4}
        return {"bytes": values + 2 * t * h * row + 8 * t, "flops": 2 * t * h * d * 2}
    by = fl = 0
    hq = case["q_heads"]
    for q, n in _lens(case):
        pairs, keys = _visible(case, q, n)
        fl += 4 * d * hq * pairs
        by += 2 * keys * h * row + 2 * q * hq * d * 2 + 4 * (-(-keys // case["page"])) + 8
        by += 4 * q * hq if case["lse"] else 0
    return {"bytes": by, "flops": fl}


# --------------------------------------------------------------------------------- inputs

def _keys_values(g, tokens, heads, d):
    """bf16 keys and values as a projection gives them, side by side in one tensor: keys with
    a few strong channels, values without."""
    kv = torch.randn((tokens, 2, heads, d), generator=g, device=DEV, dtype=torch.float32)
    strong = torch.rand((heads, d), generator=g, device=DEV) < 0.03
    kv[:, 0] *= torch.where(strong, 4.0, 0.7)
    kv[:, 1] *= 0.6
    return kv.to(torch.bfloat16)


def _slots(g, lens, page):
    """A page table [sequences][pages] with the pages in random order, the number of pages,
    and every token's slot, sequence after sequence."""
    counts = [-(-n // page) for n in lens]
    total = sum(counts) + 3
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((len(lens), max(counts)), dtype=torch.int32, device=DEV)
    slots, at = [], 0
    for b, (n, c) in enumerate(zip(lens, counts)):
        table[b, :c] = perm[at:at + c]
        s = (perm[at:at + c].to(torch.int64)[:, None] * page + torch.arange(page, device=DEV)).reshape(-1)
        slots.append(s[:n])
        at += c
    return table, total, torch.cat(slots)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    d, h, page = case["head_dim"], case["kv_heads"], case["page"]
    st = {"case": case}
    if case["op"] == "attention":
        lens = _lens(case)
        table, pages, slots = _slots(g, [n for _, n in lens], page)
        st["table"] = table
        st["kv_lens"] = torch.tensor([n for _, n in lens], dtype=torch.int32, device=DEV)
        total_q = sum(q for q, _ in lens)
        starts = [0]
        for q, _ in lens:
            starts.append(starts[-1] + q)
        st["lens"], st["starts"] = lens, starts
        st["q_starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        st["q"] = torch.randn((total_q, case["q_heads"], d), generator=g, device=DEV).to(torch.bfloat16)
    else:
        table, pages, slots = _slots(g, [case["tokens"]], page)
    data = torch.zeros((pages, h, page // 16, 18 * d + 32), dtype=torch.uint8, device=DEV)
    st["slots"] = slots
    if case["op"] == "store":
        kv = _keys_values(g, case["tokens"], h, d)
        st["k"], st["v"] = kv[:, 0], kv[:, 1]
    else:
        step = max(1, (1 << 25) // (h * d))
        for at in range(0, slots.numel(), step):
            s = slots[at:at + step]
            kv = _keys_values(g, s.numel(), h, d)
            _write(data, s, _encode(kv[:, 0]), _encode(kv[:, 1]), d)
    st["data"] = data
    if own:
        import quantized_linear_layers_block_amd as ql
        st["cache"] = ql.KVCacheNVFP4(data, pages, h, d, page)
        if case["op"] == "attention":
            nb = ql.binding.qlinear_attention_nvfp4_workspace(case["batch"], st["q"].shape[0], case["q_heads"], h, d,
                                                              case["q_len"])
            st["ws"] = torch.zeros(nb, dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------------------ plain form

def _power(e, dtype):
    """2^e for whole e, from the bits (the GPU's exp2, pow and ldexp may be an ulp off)."""
    if dtype == torch.float32:
        return ((e.to(torch.int32) + 127) << 23).view(torch.float32)
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round_even(x, step):
    return torch.round(x / step) * step   # torch.round takes ties to the even multiple


def _encode(x):
    """bf16 rows [.., D] -> E2M1 codes [.., D], E4M3 scale bytes [.., D/16], exponent bytes [..]."""
    x = x.to(torch.float32)
    mag = x.abs()
    amax = mag.amax(-1)
    m, k = torch.frexp(amax)   # amax = m 2^k, m in [1/2, 1): 2m against 2688 / 2048
    e = torch.where(m * 2 <= 1.3125, k - 1 - 11, k - 1 - 10)
    e = torch.where(amax > 0, e.clamp(-100, 117), torch.full_like(e, -100)).to(torch.int32)
    y = mag.to(torch.float64) * _power(-e, torch.float64)[..., None]
    blocks = y.reshape(*y.shape[:-1], -1, 16)
    want = blocks.amax(-1) / 6.0
    step = _power(torch.frexp(want.clamp(min=2.0 ** -6))[1] - 4, torch.float64)   # an eighth of the power of two below
    scale = _round_even(want, step).clamp(max=448.0)
    # E4M3 byte: subnormals are multiples of 2^-9, then 8 codes to each power of two
    ms, ks = torch.frexp(scale)
    byte = torch.where(scale < 2.0 ** -6, scale * 512, (ks - 1 + 7) * 8 + (ms * 2 - 1) * 8).to(torch.uint8)
    z = torch.where(scale[..., None] > 0, blocks / scale[..., None].clamp(min=2.0 ** -9), torch.zeros_like(blocks))
    # nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code
    code = torch.zeros_like(z, dtype=torch.uint8)
    for i, edge in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (z >= edge) if i % 2 else (z > edge)
    code = code.reshape(x.shape) + 8 * torch.signbit(x).to(torch.uint8)
    return code, byte, (e + 127).to(torch.uint8)


def _decode(code, byte, exp):
    """The float32 values of encoded rows (every product is exact)."""
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=code.device)
    b = byte.to(torch.float32)
    scale = torch.where(b < 8, b * 2.0 ** -9, (1 + (b % 8) / 8) * _power((byte >> 3).to(torch.int32) - 7, b.dtype))
    v = grid[code.to(torch.int64)].reshape(*byte.shape, 16) * scale[..., None]
    return v.reshape(code.shape) * _power(exp.to(torch.int32) - 127, v.dtype)[..., None]


def _parts(data, d):
    """Views of a cache's groups: K codes, scales, exps, V codes, scales, exps."""
    vb = 9 * d + 16
    lead = data.shape[:-1]
    return (data[..., :8 * d].view(*lead, 16, d // 2), data[..., 8 * d:9 * d].view(*lead, 16, d // 16),
            data[..., 9 * d:vb], data[..., vb:vb + 8 * d].view(*lead, 4, 16, d // 32, 4),
            data[..., vb + 8 * d:vb + 9 * d].view(*lead, 4, 2, d // 32, 4), data[..., vb + 9 * d:])


def _write(data, slots, k, v, d):
    pages, h, per, gb = data.shape
    kc, ks, ke, vc, vs, ve = (p for p in _parts(data.view(pages, h, per, gb), d))
    page, off = slots // (per * 16), slots % (per * 16)
    grp, t = off // 16, off % 16
    code, byte, exp = k
    kc[page, :, grp, t] = code[..., 0::2] | (code[..., 1::2] << 4)
    ks[page, :, grp, t] = byte
    ke[page, :, grp, t] = exp
    code, byte, exp = v
    pair = (code[..., 0::2] | (code[..., 1::2] << 4)).reshape(*code.shape[:-1], d // 32, 16)
    vc[page, :, grp, t // 4, :, :, t % 4] = pair.transpose(-1, -2)
    vs[page, :, grp, t // 4, :, :, t % 4] = byte.reshape(*byte.shape[:-1], d // 32, 2).transpose(-1, -2)
    ve[page, :, grp, t] = exp


def _read(data, groups, d):
    """Float32 keys and values [groups * 16][heads][D] of the listed groups (page * per + group)."""
    pages, h, per, gb = data.shape
    page, grp = groups // per, groups % per
    kc, ks, ke, vc, vs, ve = _parts(data[page, :, grp], d)   # [n, h, ...]
    n = groups.numel()
    code = torch.stack((kc & 15, kc >> 4), -1).reshape(n, h, 16, d)
    k = _decode(code, ks, ke)
    pair = vc.permute(0, 1, 2, 5, 4, 3).reshape(n, h, 16, d // 2)
    code = torch.stack((pair & 15, pair >> 4), -1).reshape(n, h, 16, d)
    v = _decode(code, vs.permute(0, 1, 2, 5, 4, 3).reshape(n, h, 16, d // 16), ve)
    return k.transpose(1, 2).reshape(n * 16, h, d), v.transpose(1, 2).reshape(n * 16, h, d)


def _plain_attention(st):
    c = st["case"]
    d, h, hq, page = c["head_dim"], c["kv_heads"], c["q_heads"], c["page"]
    grp = hq // h
    per = page // 16
    out = torch.empty_like(st["q"])
    lse = torch.empty((st["q"].shape[0], hq), dtype=torch.float32, device=out.device) if c["lse"] else None
    for b, (nq, n) in enumerate(st["lens"]):
        used = -(-n // 16)
        idx = torch.arange(used, device=out.device)
        groups = st["table"][b].to(torch.int64)[idx // per] * per + idx % per
        k, v = _read(st["data"], groups, d)
        k = k[:n].permute(1, 2, 0).contiguous()   # [h, d, n]
        v = v[:n].transpose(0, 1).contiguous()    # [h, n, d]
        r0 = st["starts"][b]
        tok = torch.arange(n, device=out.device)
        step = max(1, (1 << 28) // (n * h * grp))
        for i in range(0, nq, step):
            m = min(step, nq - i)
            q = st["q"][r0 + i:r0 + i + m].to(torch.float32).view(m, h, grp, d).transpose(0, 1)
            s = torch.matmul(q.reshape(h, m * grp, d), k) * (d ** -0.5)
            if c["causal"] and nq > 1 or c["window"]:
                pos = torch.arange(n - nq + i, n - nq + i + m, device=out.device).repeat_interleave(grp)
                hide = tok > pos[:, None]
                if c["window"]:
                    hide |= tok <= pos[:, None] - c["window"]
                s.masked_fill_(hide, -math.inf)
            top = s.amax(-1, keepdim=True)
            p = torch.exp(s - top)
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p, v) / total
            out[r0 + i:r0 + i + m] = o.view(h, m, grp, d).transpose(0, 1).reshape(m, hq, d).to(out.dtype)
            if lse is not None:
                z = (top + torch.log(total)).view(h, m, grp).transpose(0, 1)
                lse[r0 + i:r0 + i + m] = z.reshape(m, hq)
    return (out, lse) if lse is not None else out


def _plain_load(st):
    d = st["case"]["head_dim"]
    slots = st["slots"]
    pages, h, per, gb = st["data"].shape
    page, off = slots // (per * 16), slots % (per * 16)
    grp, t = off // 16, off % 16
    kc, ks, ke, vc, vs, ve = _parts(st["data"], d)
    code = torch.stack((kc[page, :, grp, t] & 15, kc[page, :, grp, t] >> 4), -1).flatten(-2)
    k = _decode(code, ks[page, :, grp, t], ke[page, :, grp, t])
    pair = vc[page, :, grp, t // 4, :, :, t % 4].transpose(-1, -2).flatten(-2)
    code = torch.stack((pair & 15, pair >> 4), -1).flatten(-2)
    byte = vs[page, :, grp, t // 4, :, :, t % 4].transpose(-1, -2).flatten(-2)
    return k.to(torch.bfloat16), _decode(code, byte, ve[page, :, grp, t]).to(torch.bfloat16)


def run(st):
    c = st["case"]
    if not own:
        if c["op"] == "attention":
            return _plain_attention(st)
        if c["op"] == "store":
            _write(st["data"], st["slots"], _encode(st["k"]), _encode(st["v"]), c["head_dim"])
        return _plain_load(st)
    import quantized_linear_layers_block_amd as ql
    if c["op"] == "attention":
        lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=DEV) if c["lse"] else None
        out = ql.attention_nvfp4(st["q"], st["cache"], st["table"], st["kv_lens"],
                                 q_starts=st["q_starts"] if c["mixed"] else None, max_q_len=c["q_len"],
                                 causal=c["causal"], window=c["window"], lse=lse, ws=st["ws"])
        return (out, lse) if c["lse"] else out
    if c["op"] == "store":
        ql.kv_store_nvfp4(st["k"], st["v"], st["slots"], st["cache"])
    return ql.kv_load_nvfp4(st["cache"], st["slots"])


# ------------------------------------------------------------------- definition, in 64 bits

def _two64(e):
    """2^e in float64 for whole e, from a table of exact powers."""
    table = torch.tensor([2.0 ** i for i in range(-160, 161)], dtype=torch.float64, device=e.device)
    return table[e.to(torch.int64) + 160]


def _value64(flat, code_at, odd, scale_at, exp_at):
    byte = flat[code_at].to(torch.int64)
    code = torch.where(odd, byte >> 4, byte & 15)
    e, m = (code >> 1) & 3, code & 1
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * _two64((e - 1).clamp(min=0)))
    s = flat[scale_at].to(torch.int64)
    se, sm = s >> 3, s & 7
    scale = torch.where(se == 0, sm / 512.0, (1 + sm / 8.0) * _two64(se - 7))
    return torch.where(code >= 8, -mag, mag) * scale * _two64(flat[exp_at].to(torch.int64) - 127)


def _rows64(data, slots, head, d, values):
    """Keys (or values) [tokens][D] of one head at the given slots, element by element from the
    address that the layout gives it."""
    pages, h, per, gb = data.shape
    base = (((slots // (16 * per)) * h + head) * per + slots % (16 * per) // 16)[:, None] * gb
    t = (slots % 16)[:, None]
    x = torch.arange(d, device=data.device)[None, :]
    odd = (x % 2 == 1).expand(slots.numel(), d)
    if not values:
        return _value64(data.view(-1), base + t * (d // 2) + x // 2, odd, base + 8 * d + t * (d // 16) + x // 16,
                        base + 9 * d + t)
    base = base + 9 * d + 16
    p, b = x // 2, x // 16
    code = base + t // 4 * (2 * d) + p % 16 * (d // 8) + p // 16 * 4 + t % 4
    scale = base + 8 * d + t // 4 * (d // 4) + b % 2 * (d // 8) + b // 2 * 4 + t % 4
    return _value64(data.view(-1), code, odd, scale, base + 9 * d + t)


def _quantised64(x):
    """The values that bf16 rows [n][D] are held as."""
    x = x.to(torch.float64)
    n, d = x.shape
    amax = x.abs().amax(1)
    e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -140) / 2688.0))
    e = torch.where(amax <= 2688.0 * _two64(e - 1), e - 1, e)   # log2 may round up past an integer
    e = torch.where(amax > 2688.0 * _two64(e), e + 1, e).clamp(-100, 117)
    unit = _two64(e)[:, None, None]
    y = x.view(n, d // 16, 16) / unit
    grid = torch.tensor([m / 512.0 for m in range(8)] + [(1 + m / 8.0) * 2.0 ** (k - 7) for k in range(1, 16)
                                                         for m in range(8)][:-1], dtype=torch.float64, device=x.device)

    def nearest(v, g):
        hi = torch.searchsorted(g, v.contiguous()).clamp(max=g.numel() - 1)
        lo = (hi - 1).clamp(min=0)
        a, b = v - g[lo], g[hi] - v
        return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)

    s = grid[nearest(y.abs().amax(2) / 6.0, grid)][:, :, None]
    fours = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    q = fours[nearest(torch.where(s > 0, y.abs() / s.clamp(min=2.0 ** -9), torch.zeros_like(y)), fours)]
    return (torch.copysign(q * s, y) * unit).view(n, d)


def exact(case, seed):
    st = prepare(case, seed)
    d, h = case["head_dim"], case["kv_heads"]
    slots = st["slots"]
    if case["op"] == "store":
        t = case["tokens"]
        return tuple(torch.cat([_quantised64(x[i:i + 4096].reshape(-1, d)) for i in range(0, t, 4096)]).view(t, h, d)
                     for x in (st["k"], st["v"]))
    if case["op"] == "load":
        return tuple(torch.stack([_rows64(st["data"], slots, i, d, values) for i in range(h)], 1)
                     for values in (False, True))
    hq, grp = case["q_heads"], case["q_heads"] // h
    total = st["q"].shape[0]
    out = torch.empty((total, hq, d), dtype=torch.float64, device=slots.device)
    lse = torch.empty((total, hq), dtype=torch.float64, device=slots.device)
    at = 0
    for b, (nq, n) in enumerate(st["lens"]):
        mine = slots[at:at + n]
        at += n
        r0 = st["starts"][b]
        for head in range(h):
            k = _rows64(st["data"], mine, head, d, False).t().contiguous()
            v = _rows64(st["data"], mine, head, d, True)
            for i in range(0, nq, 1024):
                m = min(1024, nq - i)
                for j in range(head * grp, head * grp + grp):
                    s = torch.mm(st["q"][r0 + i:r0 + i + m, j].to(torch.float64), k) / math.sqrt(d)
                    if case["causal"]:
                        last = n - nq + i + torch.arange(m, device=s.device)[:, None]
                        t = torch.arange(n, device=s.device)[None, :]
                        seen = t <= last
                        if case["window"]:
                            seen &= t > last - case["window"]
                        s = torch.where(seen, s, torch.full_like(s, -math.inf))
                    z = torch.logsumexp(s, 1)
                    out[r0 + i:r0 + i + m, j] = torch.mm(torch.exp(s - z[:, None]), v)
                    lse[r0 + i:r0 + i + m, j] = z
    return (out, lse) if case["lse"] else out
