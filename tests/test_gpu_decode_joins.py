"""GPU checks of cut sequences in the attention over the 4-bit cache: rows that are not finite keep that in their log-sum."""
import math

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


def call(mhc, ws, b, q, **k):
    return mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, want_lse=True, workspace=ws, **k)


def check_others(o, b, q, bad, scale):
    """The rows that are not in `bad` [T, Hq] are held to their bound, the others are NaN in every form."""
    assert bool(o["attn_out"][bad].isnan().all()) and bool(o["lse"][bad].isnan().all())
    off = b.offsets.tolist()
    for i, n in enumerate(b.new):
        rows = slice(off[i], off[i] + n)
        out, lse, tol, tol_lse = ref.attend(q[rows].nan_to_num(0, 0, 0), b.k[i], b.v[i], scale, "f16")
        keep = ~bad[rows]
        ref.check_out(o["attn_out"][rows][keep], out[keep], tol[keep])
        ref.check_lse(o["lse"][rows][keep], lse[keep], tol_lse[keep])


# eight warps join a row, or one (calls of more than 1,024 rows)
SHAPES = [(128, 2, 4, [40000, 300], 1), (64, 1, 7, [30000, 90], 6), (64, 8, 4, [2000 + 37 * i for i in range(40)], 1)]


@pytest.mark.parametrize("D,Hkv,G,lens,n", SHAPES)
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_query_that_is_not_finite(mhc, ws, D, Hkv, G, lens, n, value):
    """Every share's scores of its row are NaN: so are its result and its log-sum."""
    b = ref.Batch(mhc, lens, [n] * len(lens), Hkv, D, 64, seed=2)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(b.T, Hkv * G, D, generator=g, device="cuda").bfloat16()
    bad = torch.zeros(b.T, Hkv * G, dtype=torch.bool, device="cuda")
    for t, h in ((0, 0), (n - 1, G - 1), (b.T - 1, Hkv * G - 1)):
        q[t, h, 5 + h] = value
        bad[t, h] = True
    o = call(mhc, ws, b, q)
    mhc.check_status(ws)
    check_others(o, b, q, bad, D ** -0.5)


@pytest.mark.parametrize("D,Hkv,G,lens,n", SHAPES)
@pytest.mark.parametrize("table", [True, False])
def test_keys_that_are_not_there_over_whole_shares(mhc, ws, D, Hkv, G, lens, n, table):
    """Pages outside the cache, or K scales that are NaN, over many slices: the rows that see them are NaN."""
    b = ref.Batch(mhc, lens, [n] * len(lens), Hkv, D, 64, seed=3)
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(b.T, Hkv * G, D, generator=g, device="cuda").bfloat16()
    hit = 0 if len(lens) == 2 else 17
    first, last = 3, lens[hit] // 64 - 3                    # all pages but the first and the last few
    if table:
        b.page_table[hit, first:last] = b.cache.shape[0] + 5
    else:
        pages = b.page_table[hit, first:last].long()
        b.cache[pages, :, :, 8 * D:17 * D // 2] = 255
    bad = torch.zeros(b.T, Hkv * G, dtype=torch.bool, device="cuda")
    bad[hit * n:hit * n + n] = True
    check_others(call(mhc, ws, b, q), b, q, bad, D ** -0.5)
