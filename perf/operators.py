"""What the operators around the fused step are measured on: the residual addition with RMSNorm and an
MXFP8 output, the SwiGLU with an MXFP8 output, and the 8-bit matrix products that read those outputs
(one weight, or a weight per expert over ragged row groups).

``listed()`` names the cases and ``draw()`` gives more of the same ranges; ``prepare`` makes a case's
inputs from a seed, ``run`` computes it (in elementary torch operations in 32 bits, or, with ``own``
set, by the library's calls), ``exact`` gives the results in 64 bits and ``work`` the bytes and
operations a pass cannot do without.
"""
import math

import torch

own = False

EPS = 2e-6          # the norm's eps (rmsnorm_eps of the workloads)
E4M3_MAX = 448.0


def listed():
    return [
        # one speculative-verify block between two sublayers: latency only
        {"name": "norm decode", "op": "norm", "T": 6, "H": 7168, "block": 32, "mode": 0, "residual": True, "bf16": False},
        # a mid batch whose consumer takes one scale per 128 values, and whose bf16 form is wanted too
        {"name": "norm mid", "op": "norm", "T": 333, "H": 4096, "block": 128, "mode": 1, "residual": True, "bf16": True},
        # a prefill chunk
        {"name": "norm prefill", "op": "norm", "T": 8192, "H": 7168, "block": 32, "mode": 0, "residual": True, "bf16": False},
        # the experts' activations of one verify block (6 tokens, 8 experts each)
        {"name": "swiglu decode", "op": "swiglu", "T": 48, "F": 2048, "block": 32, "mode": 0},
        # the experts' activations of a prefill
        {"name": "swiglu prefill", "op": "swiglu", "T": 16384, "F": 2048, "block": 128, "mode": 0},
        # one projection of a verify block: the weight is read once, nothing else counts
        {"name": "linear decode", "op": "linear", "T": 6, "K": 7168, "N": 7168, "scales": "ue8m0", "out": "bf16"},
        # sizes that end inside a scale block and inside a tile, fp32 weight scales, an fp32 result
        {"name": "linear odd", "op": "linear", "T": 130, "K": 4064, "N": 4104, "scales": "f32", "out": "f32"},
        # a projection of a prefill chunk: the tensor cores' rate
        {"name": "linear prefill", "op": "linear", "T": 8192, "K": 7168, "N": 7168, "scales": "ue8m0", "out": "bf16"},
        # the same with a checkpoint's fp32 weight scales
        {"name": "linear prefill f32", "op": "linear", "T": 2048, "K": 7168, "N": 4096, "scales": "f32", "out": "bf16"},
        # gate and up of the experts for one verify block: most of the touched weights serve one row
        {"name": "experts decode", "op": "experts", "T": 6, "topk": 8, "E": 64, "K": 7168, "N": 4096, "gather": True, "scales": "ue8m0", "out": "bf16"},
        # gate and up of the experts for half a prefill chunk, rows taken from the layer input by index
        {"name": "experts prefill", "op": "experts", "T": 4096, "topk": 8, "E": 32, "K": 7168, "N": 4096, "gather": True, "scales": "ue8m0", "out": "bf16"},
        # down of the experts for a mid batch, rows already grouped, fp32 weight scales
        {"name": "experts down", "op": "experts", "T": 1000, "topk": 6, "E": 32, "K": 2048, "N": 7168, "gather": False, "scales": "f32", "out": "bf16"},
    ]


def _log_int(rng, lo, hi, step=1):
    """A whole multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(v / step + 0.5) * step))


def draw(rng):
    op = rng.choice(["norm", "swiglu", "linear", "linear", "experts", "experts"])
    block, mode = rng.choice([32, 128]), rng.choice([0, 1])
    if op == "norm":
        return {"op": op, "T": _log_int(rng, 1, 8192), "H": _log_int(rng, 256, 7168, 32), "block": block, "mode": mode,
                "residual": rng.random() < 0.75, "bf16": rng.random() < 0.5}
    if op == "swiglu":
        return {"op": op, "T": _log_int(rng, 1, 16384), "F": _log_int(rng, 128, 2048, 32), "block": block, "mode": mode}
    scales, out = rng.choice(["ue8m0", "f32"]), rng.choice(["bf16", "bf16", "f32"])
    if op == "linear":
        return {"op": op, "T": _log_int(rng, 1, 8192), "K": _log_int(rng, 256, 7168, 32), "N": _log_int(rng, 128, 7168, 8),
                "scales": scales, "out": out}
    E = _log_int(rng, 2, 64)
    K = _log_int(rng, 256, 7168, 32)
    N = _log_int(rng, 128, 4096, 8)
    topk = rng.randint(1, min(8, E))
    most = max(1, 32768 // (topk * max(1, E // 8)))  # the plain form pads each expert's rows to the largest group
    return {"op": op, "T": _log_int(rng, 1, min(4096, most)), "topk": topk, "E": E, "K": K, "N": N, "gather": rng.random() < 0.5,
            "scales": scales, "out": out}


# ---- the MXFP8 form: E4M3 codes and one UE8M0 scale byte per 32 values, the bytes in tiles of
# 128 rows x 4 blocks: the byte of (row m, block k) at ((m/128)*KT + k/4)*512 + (m%32)*16 + ((m%128)/32)*4 + k%4

def _tiled(s):
    """Scale bytes [M, K/32] in the tile layout (padding 0)."""
    M, KB = s.shape
    mt, kt = -(-M // 128), -(-KB // 4)
    p = torch.zeros(mt * 128, kt * 4, dtype=torch.uint8, device=s.device)
    p[:M, :KB] = s
    return p.view(mt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untiled(t, M, KB):
    mt, kt = -(-M // 128), -(-KB // 4)
    return t.view(mt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(mt * 128, kt * 4)[:M, :KB]


def _quantize(y, block, mode):
    """[M, K] fp32 -> (E4M3 codes [M, K], scale bytes [M, K/32]).  One exponent per `block` values:
    mode 0 floor(log2 amax) - 8, mode 1 the smallest E with amax <= 448 * 2^E."""
    M, K = y.shape
    nb = -(-K // block)
    a = torch.nn.functional.pad(y.abs(), (0, nb * block - K)).view(M, nb, block).amax(2)
    mant, e = torch.frexp(a.clamp(min=2.0 ** -126))           # a = mant * 2^e, mant in [0.5, 1)
    E = e - 1 - 8 + ((mant > 0.875).to(e.dtype) if mode == 1 else 0)
    E = torch.where(a < 2.0 ** -126, torch.full_like(E, -127), E.clamp(-127, 127))
    E = E.repeat_interleave(block // 32, 1)[:, : K // 32]
    q = torch.ldexp(y, -E.repeat_interleave(32, 1)).clamp(-E4M3_MAX, E4M3_MAX)
    return q.to(torch.float8_e4m3fn), (E + 127).to(torch.uint8)


def _weights(g, lead, N, K, scales, dev):
    w = torch.randn(*lead, N, K, generator=g, device=dev).mul_(112.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    sh = (*lead, -(-N // 128), -(-K // 128))
    if scales == "ue8m0":
        return w, torch.randint(127 - 13, 127 - 10, sh, generator=g, device=dev, dtype=torch.uint8)
    return w, (torch.rand(sh, generator=g, device=dev) + 0.5) * 2.0 ** -12


def _activations(g, M, K, dev):
    """Normalised activations: N(0, 1) with a few channels that stand out, in MXFP8."""
    x = torch.randn(M, K, generator=g, device=dev)
    x *= 1.0 + 15.0 * (torch.rand(K, generator=g, device=dev) < 0.01)
    q, s = _quantize(x, 32, 0)
    return q, _tiled(s)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    if c["op"] in ("norm", "swiglu"):
        M, K = c["T"], c["H"] if c["op"] == "norm" else c["F"]
        if c["op"] == "norm":
            s["x"] = torch.randn(M, K, generator=g, device=dev).bfloat16()
            if c["residual"]:
                s["residual"] = (4.0 * torch.randn(M, K, generator=g, device=dev)).bfloat16()
                s["residual_out"] = torch.empty_like(s["x"])
            s["weight"] = (1.0 + 0.1 * torch.randn(K, generator=g, device=dev)).bfloat16()
            if c["bf16"]:
                s["layer_in"] = torch.empty_like(s["x"])
        else:
            s["gate_up"] = (2.0 * torch.randn(M, 2 * K, generator=g, device=dev)).bfloat16()
        s["fp8"] = torch.empty(M, K, dtype=torch.uint8, device=dev)
        s["scales"] = torch.zeros(-(-M // 128) * 128 * (-(-K // 128) * 4), dtype=torch.uint8, device=dev)
        return s
    K, N = c["K"], c["N"]
    odt = torch.bfloat16 if c["out"] == "bf16" else torch.float32
    if c["op"] == "linear":
        s["xq"], s["xs"] = _activations(g, c["T"], K, dev)
        s["wq"], s["ws"] = _weights(g, (), N, K, c["scales"], dev)
        s["out"] = torch.empty(c["T"], N, dtype=odt, device=dev)
    else:
        T, E, topk = c["T"], c["E"], c["topk"]
        # each token takes the topk largest of E router scores; some experts are liked more
        scores = torch.randn(T, E, generator=g, device=dev) + 0.5 * torch.randn(E, generator=g, device=dev)
        ids = scores.topk(topk, 1).indices.reshape(-1)
        order = torch.argsort(ids, stable=True)
        counts = torch.bincount(ids, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
        s["most"] = int(counts.max())
        M = T * topk
        s["rows"] = (order // topk).int() if c["gather"] else None
        s["xq"], s["xs"] = _activations(g, T if c["gather"] else M, K, dev)
        s["wq"], s["ws"] = _weights(g, (E,), N, K, c["scales"], dev)
        s["out"] = torch.empty(M, N, dtype=odt, device=dev)
    s["workspace"] = torch.zeros(256, dtype=torch.uint8, device=dev)
    return s


# ---- the plain forms

def _pow2(b):
    return torch.exp2(b.float() - 127.0)


def _x32(s, K):
    q = s["xq"].float()
    return q * _pow2(_untiled(s["xs"], q.shape[0], K // 32)).repeat_interleave(32, 1)


def _w32(s, N, K):
    ws = _pow2(s["ws"]) if s["ws"].dtype == torch.uint8 else s["ws"]
    ws = ws.repeat_interleave(128, -2)[..., :N, :].repeat_interleave(128, -1)[..., :K]
    return s["wq"].float() * ws


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        x, outs = s["x"], []
        if c["residual"]:
            x = (x.float() + s["residual"].float()).bfloat16()
            outs.append(x)
        v = x.float()
        y = (v / (v.square().mean(1, keepdim=True) + EPS).sqrt() * s["weight"].float()).bfloat16()
        if c["bf16"]:
            outs.append(y)
        q, sc = _quantize(y.float(), c["block"], c["mode"])
        return outs + [q, _tiled(sc).view(torch.float8_e8m0fnu)]
    if c["op"] == "swiglu":
        a, b = s["gate_up"].float().chunk(2, 1)
        q, sc = _quantize(a / (1.0 + torch.exp(-a)) * b, c["block"], c["mode"])
        return [q, _tiled(sc).view(torch.float8_e8m0fnu)]
    N, K = c["N"], c["K"]
    odt = s["out"].dtype
    x, w = _x32(s, K), _w32(s, N, K)
    if c["op"] == "linear":
        return (x @ w.t()).to(odt)
    off, M = s["offsets"].long(), s["out"].shape[0]
    at = off[:-1, None] + torch.arange(s["most"], device=off.device)  # each expert's rows, padded to the largest group
    src = at.clamp(max=M - 1)
    src = s["rows"].long()[src] if s["rows"] is not None else src
    y = torch.bmm(x[src], w.transpose(1, 2))
    m = torch.arange(M, device=off.device)
    e = torch.bucketize(m, off[1:], right=True)
    return y[e, m - off[e]].to(odt)


def run(state):
    if not own:
        return _plain(state)
    import manifold_constrained_hyper_mhc_gb300 as mhc
    s, c = state, state["case"]
    if c["op"] == "norm":
        out = {"layer_in_fp8": s["fp8"], "layer_in_scales": s["scales"]}
        if c["residual"]:
            out["residual_out"] = s["residual_out"]
        if c["bf16"]:
            out["layer_in"] = s["layer_in"]
        o = mhc.add_rmsnorm_mxfp8(s["x"], s.get("residual"), s["weight"], rmsnorm_eps=EPS, scale_mode=c["mode"],
                                  scale_block=c["block"], want_bf16=c["bf16"], out=out)
        outs = ([o["residual_out"]] if c["residual"] else []) + ([o["layer_in"]] if c["bf16"] else [])
        return outs + [o["layer_in_fp8"].view(torch.float8_e4m3fn), o["layer_in_scales"].view(torch.float8_e8m0fnu)]
    if c["op"] == "swiglu":
        o = mhc.swiglu_mxfp8(s["gate_up"], scale_mode=c["mode"], scale_block=c["block"],
                             out={"act_fp8": s["fp8"], "act_scales": s["scales"]})
        return [o["act_fp8"].view(torch.float8_e4m3fn), o["act_scales"].view(torch.float8_e8m0fnu)]
    if c["op"] == "linear":
        return mhc.linear_mxfp8(s["xq"], s["xs"], s["wq"], s["ws"], out=s["out"], workspace=s["workspace"])
    return mhc.expert_linear_mxfp8(s["xq"], s["xs"], s["wq"], s["ws"], s["offsets"], rows=s["rows"], out=s["out"],
                                   workspace=s["workspace"])


# ---- the definition in 64 bits

def _e4m3_table(dev):
    """The 256 values of E4M3 (bias 7, no infinities, the all-ones code is NaN), from their bits."""
    v = []
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        a = math.nan if b & 127 == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-a if b & 128 else a)
    return torch.tensor(v, dtype=torch.float64, device=dev)


def _scale_at(M, KB, dev):
    """Where the tile layout holds the byte of (row, block)."""
    m, k = torch.arange(M, device=dev)[:, None], torch.arange(KB, device=dev)[None, :]
    return (m // 128 * -(-KB // 4) + k // 4) * 512 + m % 32 * 16 + m % 128 // 32 * 4 + k % 4


def _round_e4m3(v):
    """Nearest E4M3 value (ties to even), beyond the largest: the largest."""
    e = torch.frexp(v)[1].sub(1).clamp(min=-6)
    step = torch.ldexp(torch.ones_like(v), e - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_mx(y, block, mode):
    M, K = y.shape
    E = torch.empty(M, K // 32, dtype=torch.int64, device=y.device)
    for k0 in range(0, K, block):
        a = y[:, k0:k0 + block].abs().amax(1)
        e = torch.floor(torch.log2(a.clamp(min=2.0 ** -126))).long()
        e = torch.where(torch.ldexp(torch.ones_like(a), e) > a, e - 1, e)          # a log2 that rounded up
        e = torch.where(torch.ldexp(torch.ones_like(a), e + 1) <= a, e + 1, e)     # or down
        E1 = e - 8
        if mode == 1:
            E1 = E1 + (a > E4M3_MAX * torch.ldexp(torch.ones_like(a), E1)).long()
        E1 = torch.where(a < 2.0 ** -126, torch.full_like(E1, -127), E1.clamp(-127, 127))
        E[:, k0 // 32:(k0 + block) // 32] = E1[:, None]
    q = _round_e4m3(y * torch.exp2(-E.double()).repeat_interleave(32, 1))
    out = torch.full((-(-M // 128) * 128 * (-(-K // 128) * 4),), 2.0 ** -127, dtype=torch.float64, device=y.device)
    out[_scale_at(M, K // 32, y.device).reshape(-1)] = torch.exp2(E.double()).reshape(-1)
    return [q, out]


def exact(case, seed):
    s, c = prepare(case, seed), case
    dev = torch.device("cuda")
    if c["op"] == "norm":
        x, outs = s["x"].double(), []
        if c["residual"]:
            x = x + s["residual"].double()
            outs.append(x)
            x = x.float().bfloat16().double()  # the residual is held, and normalised, in bf16
        r = (x.pow(2).sum(1, keepdim=True) / c["H"] + EPS).rsqrt()
        y = x * r * s["weight"].double()
        if c["bf16"]:
            outs.append(y)
        return outs + _exact_mx(y.float().bfloat16().double(), c["block"], c["mode"])  # the bf16 layer input is quantized
    if c["op"] == "swiglu":
        a, b = s["gate_up"][:, :c["F"]].double(), s["gate_up"][:, c["F"]:].double()
        return _exact_mx(a * torch.sigmoid(a) * b, c["block"], c["mode"])
    K, N = c["K"], c["N"]
    table = _e4m3_table(dev)
    R = s["xq"].shape[0]
    xs = torch.exp2(s["xs"][_scale_at(R, K // 32, dev)].double() - 127.0)
    x = table[s["xq"].view(torch.uint8).int()] * xs.repeat_interleave(32, 1)
    n, k = torch.arange(N, device=dev)[:, None] // 128, torch.arange(K, device=dev)[None, :] // 128
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=dev)
    off = [0, R] if c["op"] == "linear" else s["offsets"].tolist()
    for e in range(len(off) - 1):
        wq, ws = (s["wq"], s["ws"]) if c["op"] == "linear" else (s["wq"][e], s["ws"][e])
        if off[e + 1] == off[e]:
            continue
        ws = torch.exp2(ws.double() - 127.0) if ws.dtype == torch.uint8 else ws.double()
        w = table[wq.view(torch.uint8).int()] * ws[n, k]
        rows = slice(off[e], off[e + 1])
        out[rows] = (x[rows] if c["op"] == "linear" or s["rows"] is None else x[s["rows"][rows].long()]) @ w.t()
    return out


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        return {"bytes": n * (2 + (4 if c["residual"] else 0) + (2 if c["bf16"] else 0) + 1 + 1 / 32) + 2 * c["H"],
                "flops": 6 * n}
    if c["op"] == "swiglu":
        n = c["T"] * c["F"]
        return {"bytes": n * (4 + 1 + 1 / 32), "flops": 8 * n}
    K, N = c["K"], c["N"]
    wscale = -(-N // 128) * -(-K // 128) * (1 if c["scales"] == "ue8m0" else 4)
    M = c["T"] if c["op"] == "linear" else c["T"] * c["topk"]
    R = c["T"] if c["op"] == "linear" or c["gather"] else M
    E = 1.0 if c["op"] == "linear" else c["E"] * (1.0 - (1.0 - c["topk"] / c["E"]) ** c["T"])  # experts that get a row
    b = R * K * (1 + 1 / 32) + E * (N * K + wscale) + M * N * (2 if c["out"] == "bf16" else 4)
    if c["op"] == "experts":
        b += (c["E"] + 1) * 4 + (4 * M if c["gather"] else 0)
    return {"bytes": b, "flops": 2.0 * M * N * K}
