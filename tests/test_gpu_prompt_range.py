"""GPU checks of the prompt attention where the sums of p v come near fp32's end."""
import pytest

torch = pytest.importorskip("torch")

import _attention as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mhc(mhc_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return mhc_lib


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rise", [3.0, 7.5, 20.0])
def test_large_values_of_v_under_scores_that_rise(mhc, D, rise):
    """v of 2^119 to 2^120 and scores that rise by 2^rise (of p) from each 128 keys to the next: the weights' sum is at most
    that of 128 equal keys and their halves' (below 2^7 * 1.2), so sums of weights, at most 1 each, with v stay below 2^128."""
    n, Hkv, G = 520, 2, 4
    g = torch.Generator(device="cuda").manual_seed(D)
    v = ((1 + torch.rand(n, Hkv, D, generator=g, device="cuda")) * 2.0 ** 119).bfloat16()
    v *= (1 - 2 * torch.randint(0, 2, v.shape, generator=g, device="cuda")).bfloat16()
    v[..., 0] = 2.0 ** 119
    k = torch.zeros(n, Hkv, D, device="cuda").bfloat16()
    k[..., 0] = (torch.arange(n, device="cuda") // 128)[:, None].bfloat16()
    q = torch.zeros(n, Hkv * G, D, device="cuda").bfloat16()
    q[..., 0] = 1.0
    scale = rise * 0.6931471805599453
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    ws = torch.zeros(mhc.prompt_workspace_size(), dtype=torch.uint8, device="cuda")
    o = mhc.prompt_attention(q, k, v, off, off, sm_scale=scale, want_lse=True, workspace=ws)
    mhc.check_status(ws)
    out, lse, tol, tol_lse = ref.attend(q, k.double(), v.double(), scale, "bf16")
    assert bool(o["attn_out"].isfinite().all())
    ref.check_out(o["attn_out"], out, tol)
    ref.check_lse(o["lse"], lse, tol_lse)
