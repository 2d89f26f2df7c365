"""GPU checks of the attention over the 4-bit cache where the 32-value blocks of a query are of very different magnitudes."""
import pytest

torch = pytest.importorskip("torch")

import _attention as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mhc(mhc_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return mhc_lib


@pytest.fixture(scope="module")
def ws(mhc):
    return torch.zeros(mhc.decode_workspace_size(), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("D,G,n", [(64, 4, 1), (64, 7, 2), (64, 8, 3), (64, 7, 6), (128, 1, 1), (128, 8, 1), (128, 4, 4), (128, 8, 3), (128, 7, 6)])
@pytest.mark.parametrize("E", [8, 21, 40])
def test_blocks_of_a_query_that_differ(mhc, ws, D, G, n, E):
    """Blocks 2^E apart, K's the other way round: every block counts the same.  (The bound: each block of a row of q keeps
    values down to 2^-20 of its largest whole and loses at most 2^-28 of that largest of the others; over 32 values of K of
    at most 6 units, that is below D 2^-23 of the block's own products' magnitudes.)"""
    Hkv, lens = 2, [700, 33, 12000]
    b = ref.Batch(mhc, lens, [n] * 3, Hkv, D, 32, seed=E)
    g = torch.Generator(device="cuda").manual_seed(G)
    q = torch.randn(b.T, Hkv * G, D // 32, 32, generator=g, device="cuda")
    up = torch.tensor([0, 1, -1, 2][:D // 32], device="cuda", dtype=torch.float64) * E
    q = (q * torch.exp2(up)[:, None]).flatten(2).bfloat16()
    for i, L in enumerate(lens):
        k = torch.randn(L, Hkv, D // 32, 32, dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(i))
        pos = torch.arange(L, device="cuda")
        ref.put(b.cache, b.page_table, i, pos, 0, *ref.quantize4((k * torch.exp2(-up)[:, None]).flatten(2), 0))
        b.k[i] = ref.get(b.cache, b.page_table, i, pos, 0)
    o = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, want_lse=True, workspace=ws)
    mhc.check_status(ws)
    for i in range(3):
        rows = slice(i * n, i * n + n)
        out, lse, tol, tol_lse = ref.attend(q[rows], b.k[i], b.v[i], D ** -0.5, "f16")
        ref.check_out(o["attn_out"][rows], out, tol)
        ref.check_lse(o["lse"][rows], lse, tol_lse)


def test_a_small_block_carries_the_score(mhc, ws):
    """q is 1 beside a block of 1.5 * 2^-27, K is 2^24 there and 0 elsewhere: scores of 32 * 1.5 / 8 = 6 for every second key, 0 for the others."""
    D, L = 128, 500
    b = ref.Batch(mhc, [L], [1], 1, D, 64, seed=1)
    k = torch.zeros(L, 1, D, dtype=torch.float64, device="cuda")
    k[::2, :, 32:64] = 2.0 ** 24
    pos = torch.arange(L, device="cuda")
    ref.put(b.cache, b.page_table, 0, pos, 0, *ref.quantize4(k, 0))
    q = torch.zeros(1, 2, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0], q[..., 32:64] = 1.0, 1.5 * 2.0 ** -27
    o = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, sm_scale=1.0, want_lse=True, workspace=ws)
    out, lse, tol, tol_lse = ref.attend(q, k, b.v[0], 1.0, "f16")
    ref.check_out(o["attn_out"], out, tol)
    ref.check_lse(o["lse"], lse, tol_lse)
