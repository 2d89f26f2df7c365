"""64-bit reference forms of the attention operators and of the 4-bit cache (torch, any device), with the bounds that
their results are held to."""
import math

import torch

import _mxfp8 as mx

E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


# ---- the cache

def quantize4(x, mode):
    """[..., D] float64 -> (codes 0..15 [..., D], scale bytes [..., D/32]); a block with a NaN: codes 0, byte 255."""
    y = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    a = y.abs().amax(-1)                                   # (torch's amax hands NaN on)
    nan = a.isnan()
    b = torch.where(nan | a.isinf(), torch.ones_like(a), a)
    mant, e = torch.frexp(b)                               # b = mant 2^e, mant in [0.5, 1)
    E = e - 3 + ((mant > 0.75).int() if mode == 1 else 0)
    E = torch.where(b < 2.0 ** -126, torch.full_like(E, -127), E.clamp(-127, 127))
    E = torch.where(a.isinf(), torch.full_like(E, 126), E)
    v = (y * mx.two_to(-E)[..., None]).abs()
    mid = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=x.device)
    q = torch.bucketize(v, mid)                            # midpoints go down ...
    up = torch.isin(v, mid[1::2])                          # ... but .75, 1.75 and 3.5 up, to the even code
    q = q + up.int()
    q = torch.where(torch.signbit(y), q + 8, q)
    q = torch.where(nan[..., None], torch.zeros_like(q), q)
    return q.reshape(x.shape).to(torch.uint8), torch.where(nan, torch.full_like(E, 128), E).add(127).to(torch.uint8)


def values4(codes, scales):
    m = E2M1.to(codes.device)[(codes & 7).int()]
    return torch.where(codes > 7, -m, m) * mx.pow2(scales).repeat_interleave(32, -1)


def code_place(D, row, d):
    """Byte of value d of row (0..15) within a part of a group, and whether it is the high half."""
    return row * (D // 2) + ((d // 32) ^ (row // (2 if D == 128 else 4)) % (D // 32)) * 16 + d % 32 // 2, d % 2


def put(cache, page_table, b, pos, part, codes, scales):
    """Writes one sequence's rows (codes [n, Hkv, D], scales [n, Hkv, D/32]) at positions pos [n] (all of them places)."""
    dev, D, page = cache.device, codes.shape[-1], cache.shape[2] * 16
    pg, at = page_table[b].long()[pos // page], pos % page
    d = torch.arange(0, D, 2, device=dev)
    byte, _ = code_place(D, (at % 16)[:, None], d[None, :])
    base = part * 17 * D // 2
    h = torch.arange(codes.shape[1], device=dev)
    cache[pg[:, None, None], h[None, :, None], (at // 16)[:, None, None], base + byte[:, None, :]] = codes[..., 0::2] | codes[..., 1::2] << 4
    sb = base + 8 * D + (at % 16)[:, None] * (D // 32) + torch.arange(D // 32, device=dev)[None, :]
    cache[pg[:, None, None], h[None, :, None], (at // 16)[:, None, None], sb[:, None, :]] = scales


def get(cache, page_table, b, pos, part):
    """float64 values [n, Hkv, D] of positions pos [n]."""
    dev, D, page = cache.device, cache.shape[3] // 17, cache.shape[2] * 16
    pg, at = page_table[b].long()[pos // page], pos % page
    base, h = part * 17 * D // 2, torch.arange(cache.shape[1], device=dev)
    byte, high = code_place(D, (at % 16)[:, None], torch.arange(D, device=dev)[None, :])
    c = cache[pg[:, None, None], h[None, :, None], (at // 16)[:, None, None], base + byte[:, None, :]]
    c = torch.where(high.bool(), c >> 4, c & 15)
    sb = base + 8 * D + (at % 16)[:, None] * (D // 32) + torch.arange(D // 32, device=dev)[None, :]
    return values4(c, cache[pg[:, None, None], h[None, :, None], (at // 16)[:, None, None], sb[:, None, :]])


class Batch:
    """A paged cache with sequences of `lens` tokens, `new` of each packed; every byte that no token owns is 255 (a NaN
    scale), and pages lie in a shuffled order with unused ones between them."""

    def __init__(self, mhc, lens, new, Hkv, D, page, seed=0, spread=0.0, k=None, dev="cuda"):
        g = torch.Generator(device=dev).manual_seed(seed)
        self.lens, self.new, self.D, self.Hkv, self.page = lens, new, D, Hkv, page
        need = [-(-n // page) for n in lens]
        P, W = sum(need) + 2, max(max(need), 1) + 1
        order = torch.randperm(P, generator=g, device=dev)
        self.page_table = torch.full((len(lens), W), -1, dtype=torch.int32, device=dev)
        self.cache = torch.full(mhc.kv_cache_shape(P, Hkv, page, D), 255, dtype=torch.uint8, device=dev)
        at = 0
        self.k, self.v = [], []
        for b, n in enumerate(lens):
            self.page_table[b, :need[b]] = order[at:at + need[b]].int()
            at += need[b]
            kv = torch.randn(2, n, Hkv, D, generator=g, device=dev, dtype=torch.float64)
            kv[0] *= 1.0 + 5.0 * (torch.rand(Hkv, D, generator=g, device=dev) < 0.03)
            if spread:
                kv *= torch.exp2(spread * torch.randn(2, n, Hkv, D // 32, generator=g, device=dev, dtype=torch.float64)).repeat_interleave(32, -1)
            pos = torch.arange(n, device=dev)
            for part, x in enumerate(kv):
                if n:
                    put(self.cache, self.page_table, b, pos, part, *quantize4(x, 0))
            self.k.append(get(self.cache, self.page_table, b, pos, 0))
            self.v.append(get(self.cache, self.page_table, b, pos, 1))
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
        self.seq_lens = i32(lens)
        self.offsets = i32([0] + torch.tensor(new).cumsum(0).tolist())
        self.T = sum(new)


# ---- attention

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 0.0}


def attend(q, k, v, scale, p_type):
    """q [n, Hq, D], the last n of the L tokens of k, v [L, Hkv, D]: (out, lse, the bound on out before its rounding, the
    bound on lse), all float64.

    The bound: each score is a sum of D products in fp32 (any order, each addition off by at most 2^-23 of the sum of
    magnitudes, truncation included), so off by D 2^-23 sum|q k| scale, and by 2^-21 of itself from the scaling and the
    exponential's own error; p_j is rounded to p_type; the sums over the keys run in fp32, n 2^-23 of the sum of
    magnitudes, with the running rescales (as many roundings again at most); l gets the same relative errors.  In fp16 p ends at
    2^-25 of 2^-11 of the largest: each of the L terms is off by at most 2^-36 of its v beside the rounding."""
    n, Hq, D = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    q = q.double()
    if L == 0:
        z = torch.zeros_like(q)
        return z, torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device), z, torch.zeros_like(z[..., 0])
    kk, vv = k.repeat_interleave(G, 1).permute(1, 0, 2), v.repeat_interleave(G, 1).permute(1, 0, 2)   # [Hq, L, D]
    qq = q.permute(1, 0, 2)
    s = qq @ kk.transpose(1, 2) * scale
    mag = qq.abs() @ kk.abs().transpose(1, 2) * abs(scale)
    hide = torch.ones(n, L, dtype=torch.bool, device=q.device).triu(L - n + 1)
    s = s.masked_fill(hide, -math.inf)
    mag = mag.masked_fill(hide, 0.0)
    m = s.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m0)
    l = p.sum(-1, keepdim=True)
    empty = (m == -math.inf)
    w = torch.where(empty, torch.zeros_like(p), p / l)
    vz = vv
    out = w @ vz
    A = w @ vz.abs()
    delta = (D * 2.0 ** -23 * mag + 2.0 ** -21 * torch.where(hide, 0.0, s).abs()).amax(-1, keepdim=True) + 2.0 ** -21
    rest = 2 * L * 2.0 ** -23
    tol = A * (U[p_type] + 2 * delta + 2 * rest) + vz.abs().amax((1, 2), keepdim=True) * (L * 2.0 ** -36 if p_type == "f16" else 2.0 ** -36)
    lse = torch.where(empty, m, m0 + l.log())[..., 0]
    tol_lse = (delta + rest)[..., 0] + 2.0 ** -21 * torch.where(empty[..., 0], 0.0, lse).abs()
    return out.permute(1, 0, 2), lse.t(), tol.permute(1, 0, 2), tol_lse.t()


def check_out(got, want, tol):
    """A bf16 result: rounded once, half a step."""
    d = (got.double() - want).abs()
    ok = d <= (tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 2.0 ** -133)
    assert bool(ok.all()), f"{int((~ok).sum())} of {ok.numel()} values off, worst {float((d / (tol + 2.0 ** -8 * want.abs() + 1e-300)).max()):.2f} of the bound"


def check_lse(got, want, tol):
    inf = want == -math.inf
    assert bool((got[inf] == -math.inf).all()) and bool(((got.double() - want).abs()[~inf] <= tol[~inf]).all())


def check_mx(codes, tiles, want, tol, mode=0):
    """MXFP8 codes [T, K] and scale tiles of want [T, K], known to tol: the exponent is that of a largest value within the
    tolerance, and each code is its value's nearest (half a step: 2^-4 of it, or half the smallest code), beyond the
    largest code the largest."""
    T, K = want.shape
    E = tiles[mx.scale_index(T, K, codes.device)].int() - 127
    a = want.abs().view(T, -1, 32)
    t = tol.view(T, -1, 32)
    lo, hi = (a - t).clamp(min=0).amax(2), (a + t).amax(2)
    assert bool(((E >= exponent(lo, mode)) & (E <= exponent(hi, mode))).all()), "scales"
    s = mx.two_to(E).repeat_interleave(32, 1)
    got = mx.e4m3_values(codes.device)[codes.int()] * s
    bound = torch.maximum((want.abs() + tol) * 2.0 ** -4, s * 2.0 ** -10) + tol + (want.abs() + tol - 448 * s).clamp(min=0)
    assert bool(((got - want).abs() <= bound * (1 + 2.0 ** -20)).all()), "codes"


def exponent(a, mode):
    mant, e = torch.frexp(a)
    E = e - 1 - 8 + ((mant > 0.875).int() if mode == 1 else 0)
    return torch.where(a < 2.0 ** -126, torch.full_like(E, -127), E.clamp(-127, 127))
