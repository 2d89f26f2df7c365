"""64-bit reference forms of the MXFP8 operators, and seeded inputs for them (torch, any device).

The scale tiles: the byte of (row m, block k of 32 values) of a [M, K] matrix is at
((m/128)*KT + k/4)*512 + (m%32)*16 + ((m%128)/32)*4 + k%4 with KT = ceil(K/128).
"""
import math

import torch

E4M3_MAX = 448.0


def scale_index(M, K, dev="cpu"):
    m, k = torch.arange(M, device=dev)[:, None], torch.arange(K // 32, device=dev)[None, :]
    return (m // 128 * ((K + 127) // 128) + k // 4) * 512 + m % 32 * 16 + m % 128 // 32 * 4 + k % 4


def scale_bytes(M, K):
    return (M + 127) // 128 * 128 * ((K + 127) // 128 * 4)


def tile_scales(s, fill=0):
    """[M, K/32] bytes -> the scale tiles, padding bytes `fill`."""
    M, K = s.shape[0], s.shape[1] * 32
    out = torch.full((scale_bytes(M, K),), fill, dtype=torch.uint8, device=s.device)
    out[scale_index(M, K, s.device).reshape(-1)] = s.reshape(-1)
    return out


def e4m3_values(dev="cpu"):
    v = []
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        a = math.nan if b & 127 == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-a if b & 128 else a)
    return torch.tensor(v, dtype=torch.float64, device=dev)


def two_to(e):
    """2^e in 64 bits for whole e in [-1022, 1023], from its bits (torch.ldexp takes its power in 32 bits, and on a
    GPU that power is not always exact)."""
    return (e.long() + 1023 << 52).view(torch.float64)


def pow2(byte):
    """2^(byte - 127) in 64 bits; the byte 255 is NaN."""
    v = two_to(byte.int() - 127)
    return torch.where(byte == 255, torch.full_like(v, math.nan), v)


def dequant_x(codes, tiles):
    M, K = codes.shape
    s = pow2(tiles[scale_index(M, K, codes.device)])
    return e4m3_values(codes.device)[codes.int()] * s.repeat_interleave(32, 1)


def dequant_w(codes, ws):
    N, K = codes.shape[-2:]
    s = pow2(ws) if ws.dtype == torch.uint8 else ws.double()
    n, k = torch.arange(N, device=codes.device) // 128, torch.arange(K, device=codes.device) // 128
    return e4m3_values(codes.device)[codes.int()] * s[..., n[:, None], k[None, :]]


def round_e4m3(v):
    """Nearest E4M3 value (ties to even), beyond the largest: the largest."""
    e = torch.frexp(v)[1].sub(1).clamp(min=-6)
    step = two_to(e - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def quantize(y, block, mode):
    """[M, K] float64 -> (values [M, K] of the codes, exponents [M, K/32])."""
    M, K = y.shape
    E = torch.empty(M, K // 32, dtype=torch.int32, device=y.device)
    for k0 in range(0, K, block):
        a = y[:, k0:k0 + block].abs().amax(1)
        mant, e = torch.frexp(a)   # a = mant 2^e, mant in [0.5, 1)
        E1 = e - 1 - 8
        if mode == 1:
            E1 = E1 + (mant > 0.875).int()
        E1 = torch.where(a < 2.0 ** -126, torch.full_like(E1, -127), E1.clamp(-127, 127))
        E[:, k0 // 32:(k0 + block) // 32] = E1[:, None]
    return round_e4m3(y * two_to(-E).repeat_interleave(32, 1)), E


def activations(M, K, seed, dev="cuda", decades=0.0):
    """MXFP8 inputs: random codes below 2^8 in magnitude, exponents over a few steps; padding scale bytes are 255
    (NaN), so that reading one shows."""
    g = torch.Generator(device=dev).manual_seed(seed)
    codes = torch.randn(M, K, generator=g, device=dev).mul_(64).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s = torch.randint(118, 124, (M, K // 32), generator=g, device=dev, dtype=torch.uint8)
    if decades:
        s = (s.int() + (torch.randn(M, 1, generator=g, device=dev) * decades).int()).clamp(1, 250).to(torch.uint8)
    return codes, tile_scales(s, 255)


def weights(lead, N, K, seed, wide, dev="cuda"):
    g = torch.Generator(device=dev).manual_seed(seed + 1000)
    codes = torch.randn(*lead, N, K, generator=g, device=dev).mul_(64).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    sh = (*lead, (N + 127) // 128, (K + 127) // 128)
    if wide:
        return codes, (torch.rand(sh, generator=g, device=dev) + 0.5) * 2.0 ** -6
    return codes, torch.randint(119, 123, sh, generator=g, device=dev, dtype=torch.uint8)
