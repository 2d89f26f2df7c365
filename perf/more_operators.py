"""What the attention operators between the 8-bit products are measured on: causal attention over packed prompts, the
4-bit (MXFP4) paged cache as it is written and read back, and the attention of new tokens over that cache.

``listed()`` names the cases and ``draw()`` gives more of the same ranges; ``prepare`` makes a case's inputs from a
seed, ``run`` computes it (in elementary torch operations in 32 bits, or, with ``own`` set, by the library's calls),
``exact`` gives the results in 64 bits and ``work`` the bytes and operations a pass cannot do without.

A batch is packed: sequence b has the rows offsets[b] .. offsets[b+1]-1 of q, k and v; they are the last tokens of the
sequence, and each attends to itself and to what is before it.  The cache is [pages, kv heads, page_size/16, 17*D] bytes:
per 16 tokens of a head the codes of K (16 rows of D/2 bytes, two E2M1 codes a byte, the even value in the low half, the
row's 16-byte chunks in the order chunk ^ ((row >> s) & (D/32-1)), s = 1 for D = 128 and 2 for D = 64), the scale bytes
of K (16 rows of D/32), then V the same way.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


def listed():
    return [
        # three short prompts in one call (one of a single token): latency only
        {"name": "prompt small", "op": "prompt", "B": 3, "nlo": 1, "nhi": 21, "plo": 0, "phi": 0, "Hq": 8, "Hkv": 2, "D": 64, "out": "bf16", "lse": True},
        # a batch of prompts of very different lengths, the result in the 8-bit form that the next product reads
        {"name": "prompt ragged", "op": "prompt", "B": 9, "nlo": 37, "nhi": 1500, "plo": 0, "phi": 0, "Hq": 32, "Hkv": 8, "D": 128, "out": "mxfp8", "lse": False},
        # one prefill chunk of a hidden size of 7168
        {"name": "prompt chunk", "op": "prompt", "B": 1, "nlo": 8192, "nhi": 8192, "plo": 0, "phi": 0, "Hq": 56, "Hkv": 8, "D": 128, "out": "bf16", "lse": False},
        # a later chunk of a long prompt: its prefix comes from the cache
        {"name": "prompt prefixed", "op": "prompt", "B": 1, "nlo": 2000, "nhi": 2000, "plo": 30001, "phi": 30001, "Hq": 56, "Hkv": 8, "D": 128, "out": "bf16", "lse": True},
        # one new token of each sequence of a batch goes to the cache, from a product's fp32 result
        {"name": "kv write decode", "op": "write", "B": 48, "nlo": 1, "nhi": 1, "plo": 0, "phi": 4000, "Hkv": 8, "D": 128, "page": 64, "dtype": "f32", "mode": 0},
        # a prefill chunk goes to the cache
        {"name": "kv write chunk", "op": "write", "B": 1, "nlo": 8192, "nhi": 8192, "plo": 4100, "phi": 4100, "Hkv": 8, "D": 128, "page": 64, "dtype": "bf16", "mode": 1},
        # a short prefix is read back
        {"name": "kv read small", "op": "read", "B": 1, "nlo": 501, "nhi": 501, "plo": 0, "phi": 0, "Hkv": 2, "D": 64, "page": 16},
        # the prefixes of four long prompts are read back for their next chunks
        {"name": "kv read prefix", "op": "read", "B": 4, "nlo": 9001, "nhi": 40000, "plo": 0, "phi": 0, "Hkv": 8, "D": 128, "page": 64},
        # one token of one sequence: latency
        {"name": "decode one", "op": "decode", "B": 1, "n": 1, "lo": 777, "hi": 777, "Hq": 8, "Hkv": 2, "D": 64, "page": 16, "out": "bf16", "lse": False},
        # a speculative-verify block of six tokens on a long sequence, the result in 8 bits
        {"name": "decode verify", "op": "decode", "B": 1, "n": 6, "lo": 32003, "hi": 32003, "Hq": 56, "Hkv": 8, "D": 128, "page": 64, "out": "mxfp8", "lse": False},
        # a serving batch of lengths from a hundred to 16,000 tokens
        {"name": "decode batch", "op": "decode", "B": 64, "n": 1, "lo": 100, "hi": 16000, "Hq": 64, "Hkv": 8, "D": 128, "page": 64, "out": "bf16", "lse": False},
        # few very long sequences, with the log-sums for a join with other keys
        {"name": "decode long", "op": "decode", "B": 3, "n": 1, "lo": 60001, "hi": 131000, "Hq": 32, "Hkv": 4, "D": 64, "page": 128, "out": "bf16", "lse": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "write", "read", "decode", "decode"])
    D, Hkv, page = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64, 128])
    G = rng.choice([1, 2, 3, 4, 7, 8, 12, 16])
    out, lse = rng.choice(["bf16", "bf16", "mxfp8"]), rng.random() < 0.3
    B = _log_int(rng, 1, 64)
    if op == "prompt":
        Hq = Hkv * min(G, 56 // Hkv)
        pairs = 8192 * 8192 * 56 / 4  # per call, with every query against every key: the plain form computes them all
        nhi = _log_int(rng, 1, min(8192, int(math.sqrt(pairs / (B * Hq)))))
        phi = 0 if rng.random() < 0.6 else _log_int(rng, 1, max(1, min(30001, int(pairs / (B * Hq * nhi)) - nhi)))
        return {"op": op, "B": B, "nlo": rng.randint(1, nhi), "nhi": nhi, "plo": rng.randint(0, phi), "phi": phi, "Hq": Hq, "Hkv": Hkv,
                "D": D, "out": out, "lse": lse}
    if op in ("write", "read"):
        nhi = _log_int(rng, 1, 98304 // B) if op == "read" else _log_int(rng, 1, 8192 // B)
        c = {"op": op, "B": B, "nlo": rng.randint(1, nhi), "nhi": nhi, "plo": 0, "phi": _log_int(rng, 1, 4100), "Hkv": Hkv, "D": D, "page": page}
        return c if op == "read" else {**c, "dtype": rng.choice(["bf16", "f32"]), "mode": rng.choice([0, 1])}
    n = rng.choice([1, 1, 2, 4, 6])
    hi = _log_int(rng, n, min(131000, 4_000_000 // (B * Hkv)))
    return {"op": op, "B": B, "n": n, "lo": rng.randint(n, hi), "hi": hi, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "page": page, "out": out, "lse": lse}


def _spread(lo, hi, B):
    """B lengths in [lo, hi], both ends among them where B > 1."""
    if B == 1:
        return [hi]
    return [lo, hi] + [lo + int((hi - lo + 1) * (b * 0.6180339887 % 1.0)) for b in range(2, B)]


def _lengths(c):
    """Each sequence's new rows and its tokens in all."""
    if c["op"] == "decode":
        return [c["n"]] * c["B"], _spread(c["lo"], c["hi"], c["B"])
    new, before = _spread(c["nlo"], c["nhi"], c["B"]), _spread(c["plo"], c["phi"], c["B"])[::-1]
    return new, [n + p for n, p in zip(new, before)]


# ---- the MXFP4 form: E2M1 codes and one UE8M0 scale byte per 32 values

def _quantize4(x, mode):
    """[..., D] fp32 -> (codes [..., D] 0..15, scale bytes [..., D/32])."""
    y = x.reshape(*x.shape[:-1], -1, 32)
    a = y.abs().amax(-1)
    mant, e = torch.frexp(a.clamp(min=2.0 ** -126))           # a = mant * 2^e, mant in [0.5, 1)
    E = e - 1 - 2 + ((mant > 0.75).to(e.dtype) if mode == 1 else 0)
    E = torch.where(a < 2.0 ** -126, torch.full_like(E, -127), E.clamp(-127, 127))
    v = torch.ldexp(y, -E[..., None])
    w = v.abs()
    q = (w > 0.25).int() + (w >= 0.75) + (w > 1.25) + (w >= 1.75) + (w > 2.5) + (w >= 3.5) + (w > 5.0)
    return (q + 8 * torch.signbit(v)).to(torch.uint8).reshape(x.shape), (E + 127).to(torch.uint8)


def _order(D, dev):
    """Where each of a row's 16-byte chunks is stored: [16 rows, D/32 chunks]."""
    r, c = torch.arange(16, device=dev)[:, None], torch.arange(D // 32, device=dev)[None, :]
    return c ^ (r >> (1 if D == 128 else 2) & D // 32 - 1)


def _groups(codes, scales):
    """Codes [..., 16, D] and scales [..., 16, D/32] of 16 tokens -> their bytes in the cache [..., 17*D/2]."""
    D = codes.shape[-1]
    b = (codes[..., 0::2] | codes[..., 1::2] << 4).reshape(*codes.shape[:-1], D // 32, 16)
    at = _order(D, codes.device)[..., None].expand(b.shape)
    b = torch.empty_like(b).scatter_(-2, at, b)
    return torch.cat([b.flatten(-3), scales.flatten(-2)], -1)


def _ungroup(b, D):
    """The cache's bytes [..., 17*D/2] of 16 tokens -> their values [..., 16, D] in fp32."""
    codes = b[..., :8 * D].reshape(*b.shape[:-1], 16, D // 32, 16)
    codes = codes.gather(-2, _order(D, b.device)[..., None].expand(codes.shape)).flatten(-2)
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], device=b.device)
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    s = torch.exp2(b[..., 8 * D:].reshape(*b.shape[:-1], 16, D // 32).float() - 127.0)
    return v * s.repeat_interleave(32, -1)


def _cached(cache, pages, D):
    """K and V [B, tokens, Hkv, D] in fp32 of the pages [B, n] of each sequence."""
    g = cache[pages.long()]                                    # [B, n, Hkv, page/16, 17 D]
    B, n, H, s, _ = g.shape
    return [_ungroup(g[..., i * 17 * D // 2:(i + 1) * 17 * D // 2], D).permute(0, 1, 3, 4, 2, 5).reshape(B, n * s * 16, H, D) for i in (0, 1)]


def _keys(g, shape, Hkv, dev):
    """Keys [.., Hkv, D] or, with their tokens in groups of 16, [.., Hkv, .., 16, D]: N(0, 1) with a few channels of
    each head that stand out."""
    at = shape.index(Hkv, 1)
    stand = [n if i in (at, len(shape) - 1) else 1 for i, n in enumerate(shape)]
    return torch.randn(*shape, generator=g, device=dev).mul_(1.0 + 5.0 * (torch.rand(stand, generator=g, device=dev) < 0.03))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c = dict(case)
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    new, lens = _lengths(c)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    cum = lambda v: i32([0] + torch.tensor(v).cumsum(0).tolist())  # noqa: E731
    T = sum(new)
    s = {"case": c, "offsets": cum(new), "seq_lens": i32(lens), "most_new": max(new), "most": max(lens), "T": T}
    if c["op"] in ("prompt", "decode"):
        s["q"] = torch.randn(T, c["Hq"], D, generator=g, device=dev).bfloat16()
        if c["out"] == "bf16":
            s["out"] = {"attn_out": torch.empty(T, c["Hq"], D, dtype=torch.bfloat16, device=dev)}
        else:
            K = c["Hq"] * D
            s["out"] = {"attn_fp8": torch.empty(T, K, dtype=torch.uint8, device=dev),
                        "attn_scales": torch.zeros(-(-T // 128) * 128 * (-(-K // 128) * 4), dtype=torch.uint8, device=dev)}
        if c["lse"]:
            s["out"]["lse"] = torch.empty(T, c["Hq"], device=dev)
    if c["op"] == "prompt":
        Tk = sum(lens)
        s["k_offsets"] = cum(lens)
        s["k"], s["v"] = _keys(g, (Tk, Hkv, D), Hkv, dev).bfloat16(), torch.randn(Tk, Hkv, D, generator=g, device=dev).bfloat16()
        s["workspace"] = torch.zeros(256, dtype=torch.uint8, device=dev)
        return s
    page = c["page"]
    width = -(-max(lens) // page)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=dev).int()
    first = torch.tensor([0] + need).cumsum(0)[:-1].to(dev)
    col = torch.arange(width, device=dev)
    at = first[:, None] + col
    s["page_table"] = torch.where(col < torch.tensor(need, device=dev)[:, None], order[at.clamp(max=pages - 1)], 0).int()
    s["page"] = page
    if c["op"] == "write":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        qkv = torch.randn(T, 3, Hkv, D, generator=g, device=dev)   # k and v are parts of a product's rows
        qkv[:, 1] = _keys(g, (T, Hkv, D), Hkv, dev)
        qkv = qkv.to(dt)
        s["k"], s["v"] = qkv[:, 1], qkv[:, 2]
        s["cache"] = torch.zeros(pages, Hkv, page // 16, 17 * D, dtype=torch.uint8, device=dev)
    else:
        s["cache"] = torch.empty(pages, Hkv, page // 16, 17 * D, dtype=torch.uint8, device=dev)
        step = max(1, (1 << 26) // (Hkv * page * D))
        for p in range(0, pages, step):
            n = min(step, pages - p)
            shape = (n, Hkv, page // 16, 16, D)
            k, v = _keys(g, shape, Hkv, dev), torch.randn(*shape, generator=g, device=dev)
            s["cache"][p:p + n] = torch.cat([_groups(*_quantize4(k, 0)), _groups(*_quantize4(v, 0))], -1)
    if c["op"] != "decode":
        s["out"] = {n: torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=dev) for n in ("k", "v")}
    else:
        s["workspace"] = torch.zeros(24 << 20, dtype=torch.uint8, device=dev)
    return s


# ---- the plain forms

def _padded(s):
    """Each sequence's rows, padded to the longest: their places among the packed rows [B, most_new], and which exist."""
    off = s["offsets"].long()
    i = torch.arange(s["most_new"], device=off.device)
    there = i < (off[1:] - off[:-1])[:, None]
    return torch.where(there, off[:-1, None] + i, 0), there


def _positions(s):
    """Of each packed row: its sequence, and its position there."""
    off = s["offsets"].long()
    t = torch.arange(s["T"], device=off.device)
    b = torch.bucketize(t, off[1:], right=True)
    return b, s["seq_lens"].long()[b] - off[b + 1] + t


def _e4m3(o):
    """[T, K] fp32 -> [E4M3 codes, scale tiles]: one exponent floor(log2 amax) - 8 per 32 values, the scale bytes in
    tiles of 128 rows x 4 blocks."""
    T, K = o.shape
    a = o.view(T, -1, 32).abs().amax(2)
    e = torch.frexp(a.clamp(min=2.0 ** -126))[1]
    E = torch.where(a < 2.0 ** -126, torch.full_like(e, -127), (e - 1 - 8).clamp(-127, 127))
    q = torch.ldexp(o, -E.repeat_interleave(32, 1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    mt, kt = -(-T // 128), -(-K // 128)
    p = torch.zeros(mt * 128, kt * 4, dtype=torch.uint8, device=o.device)
    p[:T, :K // 32] = (E + 127).to(torch.uint8)
    return [q, p.view(mt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(-1).view(torch.float8_e8m0fnu)]


def _attend(s, k, v):
    """The new rows' attention over k and v [B, most, Hkv, D] in fp32."""
    c = s["case"]
    T, Hq, Hkv, D = s["T"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    rows, there = _padded(s)
    B, n = rows.shape
    q = s["q"].float()[rows].view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    sc = q @ k.permute(0, 2, 3, 1)
    sc *= D ** -0.5
    off = s["offsets"].long()
    sees = s["seq_lens"].long()[:, None] - (off[1:] - off[:-1])[:, None] + torch.arange(n, device=off.device) + 1   # keys of each row
    hide = torch.arange(k.shape[1], device=off.device) >= sees.repeat_interleave(G, 1)[:, None, :, None]
    sc.masked_fill_(hide, -math.inf)
    del hide
    m = sc.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    sc -= m
    sc.exp_()
    l = sc.sum(-1, keepdim=True)
    o = (sc @ v.permute(0, 2, 1, 3)) / l
    pick = lambda x: x.view(B, Hkv, n, G, -1).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, -1)[there]  # noqa: E731
    o = pick(o)
    outs = [o.bfloat16()] if c["out"] == "bf16" else _e4m3(o.reshape(T, Hq * D))
    return outs + ([pick(m + l.log()).view(T, Hq)] if c["lse"] else [])


def _plain(s):
    c = s["case"]
    if c["op"] == "prompt":
        off = s["k_offsets"].long()
        i = torch.arange(s["most"], device=off.device)
        there = i < (off[1:] - off[:-1])[:, None]
        rows = torch.where(there, off[:-1, None] + i, 0)
        return _attend(s, s["k"].float()[rows], s["v"].float()[rows])
    if c["op"] == "decode":
        return _attend(s, *_cached(s["cache"], s["page_table"], c["D"]))
    D, page = c["D"], c["page"]
    b, pos = _positions(s)
    p, r = s["page_table"].long()[b, pos // page], pos % page
    if c["op"] == "write":
        q, e = _quantize4(torch.stack([s["k"], s["v"]], 1).float(), c["mode"])           # [T, 2, Hkv, D]
        q = (q[..., 0::2] | q[..., 1::2] << 4).unflatten(-1, (D // 32, 16))
        at = _order(D, p.device)[r % 16][:, None, None, :, None].expand(q.shape)
        q = torch.empty_like(q).scatter_(3, at, q).flatten(3)
        half = s["cache"].unflatten(3, (2, 17 * D // 2))                                 # [pages, Hkv, page/16, 2, ..]
        half[..., :8 * D].unflatten(-1, (16, D // 2))[p, :, r // 16, :, r % 16] = q.transpose(1, 2)
        half[..., 8 * D:].unflatten(-1, (16, D // 32))[p, :, r // 16, :, r % 16] = e.transpose(1, 2)
    g = s["cache"][p, :, r // 16]                               # each row's group of 16 tokens [T, Hkv, 17 D]
    t = torch.arange(s["T"], device=p.device)
    return [_ungroup(x, D)[t, :, r % 16].bfloat16() for x in g.split(17 * D // 2, -1)]


def run(state):
    if not own:
        return _plain(state)
    import manifold_constrained_hyper_mhc_gb300 as mhc
    s, c = state, state["case"]
    if c["op"] == "write":
        mhc.kv_write_mxfp4(s["k"], s["v"], s["cache"], s["page_table"], s["seq_lens"], s["offsets"], scale_mode=c["mode"])
    if c["op"] in ("write", "read"):
        o = mhc.kv_read_mxfp4(s["cache"], s["page_table"], s["seq_lens"], s["offsets"], out=s["out"])
        return [o["k"], o["v"]]
    form = {"sm_scale": c["D"] ** -0.5, "want_bf16": c["out"] == "bf16", "want_mxfp8": c["out"] == "mxfp8", "want_lse": c["lse"],
            "out": s["out"], "workspace": s["workspace"]}
    if c["op"] == "prompt":
        o = mhc.prompt_attention(s["q"], s["k"], s["v"], s["offsets"], s["k_offsets"], **form)
    else:
        o = mhc.decode_attention_mxfp4(s["q"], s["cache"], s["page_table"], s["seq_lens"], s["offsets"], **form)
    outs = [o["attn_out"]] if c["out"] == "bf16" else [o["attn_fp8"].view(torch.float8_e4m3fn), o["attn_scales"].view(torch.float8_e8m0fnu)]
    return outs + ([o["lse"]] if c["lse"] else [])


# ---- the definition in 64 bits

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _cache_values(cache, page_table, length, b, part, D):
    """[length, Hkv, D] of sequence b: K (part 0) or V (part 1), byte by byte from the layout's rule."""
    dev, page = cache.device, cache.shape[2] * 16
    pos = torch.arange(length, device=dev)
    g = cache[page_table[b].long()[pos // page], :, pos % page // 16]           # [length, Hkv, 17 D]
    r, d, base = (pos % 16)[:, None], torch.arange(D, device=dev)[None, :], part * 17 * D // 2
    chunk = d // 32 ^ (r // (2 if D == 128 else 4)) % (D // 32)
    byte = (base + r * (D // 2) + chunk * 16 + d % 32 // 2)[:, None, :].expand(-1, g.shape[1], -1)
    code = g.gather(2, byte).int() >> (d % 2 * 4)[None] & 15
    scale = g.gather(2, (base + 8 * D + r * (D // 32) + d // 32)[:, None, :].expand(-1, g.shape[1], -1))
    mag = torch.tensor(E2M1, dtype=torch.float64, device=dev)[code & 7]
    return torch.where(code > 7, -mag, mag) * torch.exp2(scale.double() - 127.0)


def _to_values4(x, mode):
    """The values that x [..., D] in 64 bits stands for after it is held in MXFP4."""
    out = torch.empty_like(x)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    for d in range(0, x.shape[-1], 32):
        y = x[..., d:d + 32]
        a = y.abs().amax(-1, keepdim=True)
        E = torch.floor(torch.log2(a.clamp(min=2.0 ** -126)))
        E = torch.where(torch.exp2(E) > a, E - 1, E)
        E = torch.where(torch.exp2(E + 1) <= a, E + 1, E) - 2
        if mode == 1:
            E = E + (a > 6.0 * torch.exp2(E)).double()
        E = torch.where(a < 2.0 ** -126, torch.full_like(E, -127.0), E.clamp(-127, 127))
        v = (y.abs() * torch.exp2(-E)).clamp(max=6.0)
        hi = torch.bucketize(v, grid).clamp(max=7)                              # the first value >= v
        lo = (hi - 1).clamp(min=0)
        up, down = grid[hi] - v, v - grid[lo]
        at = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)  # the nearer one, or the even code
        out[..., d:d + 32] = torch.copysign(grid[at], y) * torch.exp2(E)
    return out


def _exact_e4m3(o):
    """What the E4M3 codes of o stand for, before their rounding.  The scales are a choice, not a computed number: where
    a block's largest value lies at a power of two, either exponent is right."""
    T, K = o.shape
    a = o.view(T, K // 32, 32).abs().amax(2)
    E = torch.floor(torch.log2(a.clamp(min=2.0 ** -126)))
    E = torch.where(torch.exp2(E) > a, E - 1, E)
    E = torch.where(torch.exp2(E + 1) <= a, E + 1, E) - 8
    E = torch.where(a < 2.0 ** -126, torch.full_like(E, -127.0), E.clamp(-127, 127))
    return [(o * torch.exp2(-E).repeat_interleave(32, 1)).clamp(-E4M3_MAX, E4M3_MAX), None]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    D, Hkv = c["D"], c["Hkv"]
    if c["op"] == "write":
        return [_to_values4(s[n].double(), c["mode"]) for n in ("k", "v")]
    new, lens = _lengths(c)
    if c["op"] == "read":
        return [torch.cat([_cache_values(s["cache"], s["page_table"], L, b, part, D)[L - n:] for b, (n, L) in enumerate(zip(new, lens))]) for part in (0, 1)]
    G = c["Hq"] // Hkv
    out = torch.empty(s["T"], c["Hq"], D, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["T"], c["Hq"], dtype=torch.float64, device="cuda")
    t0 = k0 = 0
    for b, (n, L) in enumerate(zip(new, lens)):
        if c["op"] == "prompt":
            k, v = s["k"][k0:k0 + L].double(), s["v"][k0:k0 + L].double()
        else:
            k, v = (_cache_values(s["cache"], s["page_table"], L, b, part, D) for part in (0, 1))
        hide = torch.ones(n, L, dtype=torch.bool, device="cuda").triu_(L - n + 1)
        for h in range(c["Hq"]):
            z = s["q"][t0:t0 + n, h].double() @ k[:, h // G].t() / math.sqrt(D)
            z.masked_fill_(hide, -math.inf)
            lse[t0:t0 + n, h] = torch.logsumexp(z, 1)
            out[t0:t0 + n, h] = torch.softmax(z, 1) @ v[:, h // G]
        t0, k0 = t0 + n, k0 + L
    outs = [out] if c["out"] == "bf16" else _exact_e4m3(out.view(s["T"], -1))
    return outs + ([lse] if c["lse"] else [])


def work(case):
    c = case
    new, lens = _lengths(c)
    T, Hkv, D = sum(new), c["Hkv"], c["D"]
    held = Hkv * 2 * D * 17 / 32                                # bytes of a token in the cache
    if c["op"] == "write":   # and read back, as this file's pass does
        return {"bytes": T * (2 * Hkv * D * (2 if c["dtype"] == "bf16" else 4) + 2 * held + 2 * Hkv * D * 2), "flops": 8 * T * Hkv * D}
    if c["op"] == "read":
        return {"bytes": T * (held + 2 * Hkv * D * 2), "flops": 2 * T * Hkv * D}
    pairs = sum(n * (L - n) + n * (n + 1) // 2 for n, L in zip(new, lens))
    row = c["Hq"] * D * (2 + (2 if c["out"] == "bf16" else 33 / 32)) + (4 * c["Hq"] if c["lse"] else 0)
    keys = sum(lens) * (held if c["op"] == "decode" else 2 * Hkv * D * 2)
    return {"bytes": T * row + keys, "flops": 4.0 * D * c["Hq"] * pairs}
