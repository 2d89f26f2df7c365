"""GPU tests of add_rmsnorm_mxfp8 where fp32 leaves its range: rows whose mean square fp32 does not hold, with eps 0 or
next to nothing.

Tolerance: half a bf16 step (2^-8) of a value that is off by at most 2^-20 before it (half the relative error of the square
sum, at most 31 additions and products of 2^-24 in a row, and two roundings), and half a step of bf16's smallest values,
2^-134, plus what fp32 drops of a product below its range, 2^-150 times a root of at most 2^20.  Asked:
(2^-8 + 2^-19) |y| + 2^-129."""
import pytest

torch = pytest.importorskip("torch")

import _mxfp8 as ref  # noqa: E402
from test_gpu_norm_mxfp8 import check_mx, norm_ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mhc(mhc_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return mhc_lib


MAGNITUDES = [2e-40, 1e-38, 1e-30, 1e-25, 1e-23, 1e-21, 1e-20, 5e-20, 6e-20, 1e-19, 1e-13, 1e-6, 1.0, 1e6, 1e9, 1e15, 1e18, 2e19,
              1e20, 1e25, 1e30, 1e38, 3e38]


def rows_of(magnitudes, T, H, seed):
    """Rows whose values are between half a magnitude and the magnitude, of both signs (bf16 holds them all)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    m = torch.tensor(magnitudes, dtype=torch.float64, device="cuda").repeat(T // len(magnitudes) + 1)[:T, None]
    x = (0.5 + 0.5 * torch.rand(T, H, generator=g, device="cuda").double()) * m
    x = torch.where(torch.rand(T, H, generator=g, device="cuda") < 0.5, -x, x).float().bfloat16()
    return x, (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).bfloat16()


def close(got, want):
    return (got.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -19) * want.abs() + 2.0 ** -129


@pytest.mark.parametrize("block,mode", [(32, 0), (128, 1)])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-38, 2e-6])
@pytest.mark.parametrize("H", [32, 992, 1024, 2048, 4096, 7168, 8192, 8224, 65536])
def test_rows_of_any_magnitude(mhc, H, eps, block, mode):
    x, w = rows_of(MAGNITUDES, len(MAGNITUDES), H, H)
    o = mhc.add_rmsnorm_mxfp8(x, None, w, rmsnorm_eps=eps, scale_mode=mode, scale_block=block, want_bf16=True)
    want = norm_ref(x, w, torch.tensor(eps, dtype=torch.float32).double().item())  # the eps that the call gets
    bad = ~close(o["layer_in"], want)
    assert not bool(bad.any()), [(MAGNITUDES[t], o["layer_in"][t, 0].item(), want[t, 0].item()) for t in bad.any(1).nonzero().flatten().tolist()]
    check_mx(o["layer_in_fp8"], o["layer_in_scales"], o["layer_in"].double(), block, mode)


@pytest.mark.parametrize("T,H", [(9001, 512), (1003, 7168), (700, 8224)])
def test_far_rows_among_others_in_turn(mhc, T, H):
    """More rows than run at once, the far ones in no fixed place of a CTA's turn, the residual updated in place; the
    ordinary rows are those of a call without the far ones, bit for bit."""
    x, w = rows_of([1.0, 1e-22, 3.0, 0.1, 1e22, 1e25, 2.0], T, H, 5)
    plain = x.abs().amax(1)
    plain = (plain > 1e-3) & (plain < 1e3)
    r = torch.zeros_like(x)
    o = mhc.add_rmsnorm_mxfp8(x, r, w, rmsnorm_eps=0.0, want_bf16=True, out={"residual_out": r})
    assert o["residual_out"] is r and torch.equal(r, x)
    assert bool(close(o["layer_in"], norm_ref(x, w, 0.0)).all())
    few = mhc.add_rmsnorm_mxfp8(x[plain].contiguous(), None, w, rmsnorm_eps=0.0, want_bf16=True)
    assert torch.equal(few["layer_in"].view(torch.int16), o["layer_in"][plain].view(torch.int16))
    assert torch.equal(few["layer_in_fp8"], o["layer_in_fp8"][plain])


@pytest.mark.parametrize("H", [1024, 8224])
def test_rows_without_a_norm(mhc, H):
    """Zeros with eps 0 have no norm (0 / 0); infinities and NaN as in the formula; the rows beside them are untouched by it."""
    x, w = rows_of([1.0], 6, H, 7)
    x[1] = 0
    x[2, 3] = float("inf")
    x[3, H - 1] = float("-inf")
    x[4, 9] = float("nan")
    o = mhc.add_rmsnorm_mxfp8(x, None, w, rmsnorm_eps=0.0, want_bf16=True)
    y = o["layer_in"]
    want = norm_ref(x, w, 0.0)
    assert torch.equal(y.isnan(), want.isnan())
    assert bool(y[1].isnan().all()) and bool(y[4].isnan().all()) and int(y[2].isnan().sum()) == 1 and int(y[3].isnan().sum()) == 1
    assert bool((y[2:4].nan_to_num() == 0).all())
    assert bool(close(y[[0, 5]], want[[0, 5]]).all())


def test_rows_at_the_borders_do_not_depend_on_the_rows_beside_them(mhc):
    """Rows whose mean square is near 2^-40 or 2^60 (where fp64 begins) have the same bits alone and in turn with far ones."""
    T, H = 9001, 512
    edge = [2.0 ** p * f for p in (-20, 30) for f in (0.99, 0.995, 0.999, 1.0, 1.001, 1.005, 1.01)]
    g = torch.Generator(device="cuda").manual_seed(3)
    m = torch.tensor([*edge, 1e-24, 1e24, 1.0], dtype=torch.float64, device="cuda").repeat(T // 17 + 1)[:T, None]
    x = torch.randn(T, H, generator=g, device="cuda").double()
    x = (x / x.square().mean(1, keepdim=True).sqrt() * m).float().bfloat16()
    w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).bfloat16()
    o = mhc.add_rmsnorm_mxfp8(x, None, w, rmsnorm_eps=0.0, want_bf16=True)
    assert bool(close(o["layer_in"], norm_ref(x, w, 0.0)).all())
    ordinary = (m[:, 0] > 1e-9) & (m[:, 0] < 1e12)
    for pick in (ordinary, ordinary & (torch.arange(T, device="cuda") < 400)):
        few = mhc.add_rmsnorm_mxfp8(x[pick].contiguous(), None, w, rmsnorm_eps=0.0, want_bf16=True)
        assert torch.equal(few["layer_in"].view(torch.int16), o["layer_in"][pick].view(torch.int16))
        assert torch.equal(few["layer_in_fp8"], o["layer_in_fp8"][pick])
