"""GPU checks of cut sequences in the attention over the 4-bit cache: rows that are not finite keep that in their
log-sum, and no part of a sequence is lost, taken twice or put elsewhere."""
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


def fill(b, i, k, v):
    pos = torch.arange(b.lens[i], device="cuda")
    for part, x in enumerate((k, v)):
        ref.put(b.cache, b.page_table, i, pos, part, *ref.quantize4(x, 0))
    b.k[i], b.v[i] = (ref.get(b.cache, b.page_table, i, pos, p) for p in (0, 1))


@pytest.mark.parametrize("D,Hkv,G,lens,n", [(128, 1, 8, [40000], 1), (64, 2, 4, [70001, 500], 1), (128, 2, 3, [20000, 1, 9000, 64, 12345], 5), (64, 1, 24, [33333], 1),
                                            (128, 1, 7, [16001], 6), (64, 8, 4, [2000 + 37 * i for i in range(40)], 1)])
def test_every_slice_is_summed_once(mhc, ws, D, Hkv, G, lens, n):
    """Equal scores (q of zeros), and V that is 1 in the column of its slice of 32 tokens: a result is its columns' share of
    the tokens.  p is a power of two and the sums are whole multiples of it below 2^24 of them: exact.  What is rounded is
    the division, the means' weights in the join (a share's count over the sum of counts so far; its factor is rounded
    twice, the product and the addition once each, of at most 1,824 parts that are all below the result) and the result."""
    b = ref.Batch(mhc, lens, [min(n, L) for L in lens], Hkv, D, 64, seed=4)
    for i, L in enumerate(lens):
        j = torch.arange(L, device="cuda")
        v = torch.nn.functional.one_hot(j // 32 % D, D).double()[:, None, :].repeat(1, Hkv, 1)
        for h in range(Hkv):
            v[:, h] = v[:, h].roll(h, 1)                    # (a head's columns are its own)
        fill(b, i, torch.randn(L, Hkv, D, dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(i)), v)
        assert torch.equal(b.v[i], v)
    q = torch.zeros(b.T, Hkv * G, D, dtype=torch.bfloat16, device="cuda")
    o = call(mhc, ws, b, q)
    t = 0
    for i, L in enumerate(lens):
        for r in range(b.new[i]):
            sees = L - b.new[i] + r + 1
            want = (b.v[i][:sees].sum(0) / sees).repeat_interleave(G, 0)
            d = (o["attn_out"][t].double() - want).abs()
            assert bool((d <= want * (2.0 ** -8 + 1824 * 4 * 2.0 ** -24)).all())
            # log2 of the sum (2 ulp), plus m, times ln 2: three roundings of at most 2^-23 of 32
            assert float((o["lse"][t].double() - math.log(sees)).abs().max()) <= 5 * 2.0 ** -23 * 32
            t += 1


@pytest.mark.parametrize("D,Hkv,G,L", [(128, 8, 8, 40000), (128, 2, 64, 30011), (64, 1, 48, 52000), (64, 4, 16, 9000), (128, 4, 1, 25000)])
def test_one_key_of_every_share(mhc, ws, D, Hkv, G, L):
    """Each head looks for one key, all of them spread over the line: its result is that key's V."""
    b = ref.Batch(mhc, [L], [1], Hkv, D, 32, seed=5)
    at = torch.linspace(0, L - 1, Hkv * G, device="cuda").round().long().view(G, Hkv)   # (neighbours in different heads)
    k = torch.zeros(L, Hkv, D, dtype=torch.float64, device="cuda")
    q = torch.zeros(1, Hkv * G, D, dtype=torch.bfloat16, device="cuda")
    for h in range(Hkv):
        for g in range(G):
            k[at[g, h], h, g] = 4.0
            q[0, h * G + g, g] = 16.0
    v = torch.randn(L, Hkv, D, dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(6))
    fill(b, 0, k, v)
    o = call(mhc, ws, b, q, sm_scale=1.0)
    for h in range(Hkv):
        want = b.v[0][at[:, h], h]
        # the others' weight: L e^-64, below 2^-70
        got = o["attn_out"][0, h * G:h * G + G].double()
        assert bool(((got - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -10) + 2.0 ** -60).all())   # (P' is a power of two or a half's rounding of it: 2^-11)
    # m is 64 log2 e in fp32 (2^-17.5 a step), times ln 2
    assert float((o["lse"].double() - 64.0).abs().max()) <= 4 * 2.0 ** -18
