"""GPU tests of swiglu_mxfp8 at the ends of fp32's range, against the 64-bit definition: block maxima next to a border between
two exponents down to the smallest exponent.

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
