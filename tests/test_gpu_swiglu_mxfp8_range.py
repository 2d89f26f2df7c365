"""GPU tests of swiglu_mxfp8 at the ends of fp32's range, against the 64-bit definition: block maxima next to a border between
two exponents down to the smallest exponent, and products beyond fp32's largest value.

No tolerance: the scale bytes are exact, and the codes are those of the exact value where that is a normal E4M3 number (below,
off by one step of 2^-9 at most)."""
import pytest

torch = pytest.importorskip("torch")

import _mxfp8 as ref  # noqa: E402
from test_gpu_norm_mxfp8 import check_mx  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mhc(mhc_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return mhc_lib


def exact(gu):
    a, b = gu.double().chunk(2, 1)
    return a / (1 + torch.exp(-a)) * b


@pytest.mark.parametrize("block,mode", [(32, 0), (32, 1), (128, 0), (128, 1)])
def test_maxima_next_to_a_border_of_small_exponents(mhc, block, mode):
    """silu(a) b with a = -+2^-k lies just below or above a / 2 b, which is a power of two, or 1.75 times one."""
    F = 128
    top = [(s * 2.0 ** -k, f * 2.0 ** (p + k + 1)) for s in (-1, 1) for k in (4, 9, 14, 19, 22, 25, 28) for f in (1.0, 1.75)
           for p in range(-126, -99)]
    top = torch.tensor(top, dtype=torch.float64)
    T = len(top)
    gen = torch.Generator().manual_seed(1)
    at = torch.randint(0, F, (T,), generator=gen)
    gate = torch.rand(T, F, generator=gen, dtype=torch.float64) * top[:, :1]          # the others are smaller
    up = top[:, 1:] * torch.rand(T, F, generator=gen, dtype=torch.float64) * 0.9
    t = torch.arange(T)
    gate[t, at], up[t, at] = top[:, 0], top[:, 1]
    gu = torch.cat([gate, up], 1).bfloat16().cuda()
    assert torch.equal(gu[t, at].double().cpu(), top[:, 0])
    o = mhc.swiglu_mxfp8(gu, scale_mode=mode, scale_block=block)
    check_mx(o["act_fp8"], o["act_scales"], exact(gu), block, mode, exact_subnormals=False)


@pytest.mark.parametrize("block,mode", [(32, 0), (32, 1), (128, 0), (128, 1)])
def test_products_beyond_fp32(mhc, block, mode):
    """Products from 2^118 to 2^150 in one block: the exponent is the largest one's (at most 127), every code its own."""
    T, F = 400, 256
    gen = torch.Generator().manual_seed(2)
    top = 118 + torch.randint(0, 33, (T, 1), generator=gen)
    e = top - torch.randint(0, 20, (T, F), generator=gen)
    ga = torch.randint(7, 100, (T, F), generator=gen)
    ga = torch.minimum(ga, e)
    sig = lambda: 1 + torch.randint(0, 128, (T, F), generator=gen).double() / 128
    sign = torch.where(torch.rand(T, F, generator=gen) < 0.5, -1.0, 1.0).double()
    gate, up = sig() * ref.two_to(ga), sig() * ref.two_to(e - ga).clamp(max=2.0 ** 126) * sign
    gu = torch.cat([gate, up], 1).bfloat16().cuda()
    assert bool(gu.isfinite().all())
    want = exact(gu)
    assert bool((want.abs() > 2.0 ** 128).any(1).sum() > T // 2)
    o = mhc.swiglu_mxfp8(gu, scale_mode=mode, scale_block=block)
    check_mx(o["act_fp8"], o["act_scales"], want, block, mode, exact_subnormals=False)


@pytest.mark.parametrize("block", [32, 128])
def test_an_infinite_product_gives_its_block_the_exponent_120(mhc, block):
    F = 128
    gate, up = torch.full((3, F), 2.0 ** 64), torch.full((3, F), 2.0 ** 50)
    gate[0, 5] = float("inf")
    up[1, 100] = float("-inf")
    up[2, 33] = float("inf")
    up[:, 32:40:2] *= 2.0 ** 13   # 2^127
    up[:, 64:72:2] *= 2.0 ** 14   # 2^128
    up[:, 96:99] *= 2.0 ** 15     # 2^129 = 512 2^120: the largest code
    gu = torch.cat([gate, up], 1).bfloat16().cuda()
    o = mhc.swiglu_mxfp8(gu, scale_block=block)
    want = exact(gu)
    has = want.isinf().view(3, F // block, block).any(2).repeat_interleave(block // 32, 1)
    E = o["act_scales"][ref.scale_index(3, F, "cuda")].int() - 127
    assert bool((E[has] == 120).all())
    vals = ref.e4m3_values("cuda")[o["act_fp8"].int()]
    in_it = has.repeat_interleave(32, 1)
    assert torch.equal(vals[in_it], ref.round_e4m3((want * 2.0 ** -120).clamp(-1e6, 1e6))[in_it])
