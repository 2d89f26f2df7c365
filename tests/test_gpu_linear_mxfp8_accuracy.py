"""GPU tests of the 8-bit products' accuracy as a whole, and of weight scales that are not finite.

The elementwise tests hold each result to its worst case, K 2^-23 sum |x w|, which at large K is several products wide.  Here
the inputs have signs at random, so sums and errors grow like roots.  The tensor cores add 32 products at a time to an fp32
sum: n = K / 32 additions (and, with fp32 weight scales, one rounding and one addition per 128), each off by at most one unit,
2^-23 of the partial sum, which after j of them is sqrt(j / n) of the result's root mean square.  With errors of either sign
the result is off by 2^-23 sqrt((n + 1) / 2 + n / 4) of it in the root mean square, and an element by eight times that (a
million elements of a normal distribution stay within five).  The fp32 scale of a block is applied with one rounding more:
n / 4 of them, counted above.  A product that is lost is about 1 / sqrt(K) of the result: thousands of times that."""
import math

import pytest

torch = pytest.importorskip("torch")

import _mxfp8 as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mhc(mhc_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return mhc_lib


@pytest.fixture(scope="module")
def ws(mhc):
    return torch.zeros(mhc.linear_workspace_size(), dtype=torch.uint8, device="cuda")


def even_activations(T, K, seed):
    """Codes of one distribution under one exponent: every product counts about alike."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randn(T, K, generator=g, device="cuda").mul_(64).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, ref.tile_scales(torch.full((T, K // 32), 121, dtype=torch.uint8, device="cuda"), 255)


def even_weights(lead, N, K, seed, wide):
    codes, s = ref.weights(lead, N, K, seed, wide)
    return codes, (s if wide else torch.full_like(s, 121))


def rms(v):
    return v.square().mean().sqrt().item()


def hold(got, x, w):
    K = x.shape[1]
    want = x @ w.t()
    scale = want.square().mean(1, keepdim=True).sqrt()   # a row's size
    err = (got.double() - want) / scale
    n = K / 32
    bound = 2.0 ** -23 * math.sqrt((n + 1) / 2 + n / 4)
    assert rms(err) <= bound, (rms(err), bound)
    assert err.abs().max().item() <= 8 * bound, (err.abs().max().item(), bound)


@pytest.mark.parametrize("wide", [False, True], ids=["ue8m0", "f32scale"])
@pytest.mark.parametrize("T,K,N", [(6, 7168, 4096), (40, 16384, 1024), (130, 4064, 2056), (128, 7168, 2048), (700, 7168, 4096), (2048, 2080, 4096)])
def test_linear_errors_grow_like_roots(mhc, ws, T, K, N, wide):
    xq, xs = even_activations(T, K, T + K)
    wq, wsc = even_weights((), N, K, N, wide)
    out = mhc.linear_mxfp8(xq, xs, wq, wsc, out_dtype=torch.float32, workspace=ws)
    mhc.check_status(ws)
    hold(out, ref.dequant_x(xq, xs), ref.dequant_w(wq, wsc))


@pytest.mark.parametrize("wide", [False, True], ids=["ue8m0", "f32scale"])
@pytest.mark.parametrize("gather", [False, True])
def test_expert_errors_grow_like_roots(mhc, ws, gather, wide):
    M, E, K, N, R = 1500, 6, 7168, 1032, 400
    xq, xs = even_activations(R if gather else M, K, 3)
    wq, wsc = even_weights((E,), N, K, 4, wide)
    g = torch.Generator().manual_seed(5)
    rows = torch.randint(0, R, (M,), generator=g).int().cuda() if gather else None
    o = [0, 1, 300, 300, 850, 1499, M]
    out = mhc.expert_linear_mxfp8(xq, xs, wq, wsc, torch.tensor(o, dtype=torch.int32, device="cuda"), rows=rows,
                                  out_dtype=torch.float32, workspace=ws)
    mhc.check_status(ws)
    x = ref.dequant_x(xq, xs)
    x = x[rows.long()] if gather else x
    for e in range(E):
        if o[e + 1] > o[e]:
            hold(out[o[e]:o[e + 1]], x[o[e]:o[e + 1]], ref.dequant_w(wq[e], wsc[e]))


@pytest.mark.parametrize("T,N", [(3, 392), (200, 520), (4100, 4104)])
def test_a_nan_weight_scale_stays_in_its_128_columns(mhc, ws, T, N):
    K = 416
    xq, xs = ref.activations(T, K, 5)
    for wide, bad in ((False, 255), (True, float("nan"))):
        wq, wsc = ref.weights((), N, K, 6, wide)
        wsc[1, 2] = bad
        out = mhc.linear_mxfp8(xq, xs, wq, wsc, out_dtype=torch.float32, workspace=ws)
        eq, es = torch.stack([wq, wq]), torch.stack([wsc, wsc])
        es[0, 1, 2] = es[0, 0, 0]
        two = mhc.expert_linear_mxfp8(xq, xs, eq, es, torch.tensor([0, T // 2, T], dtype=torch.int32, device="cuda"),
                                      out_dtype=torch.float32, workspace=ws)
        mhc.check_status(ws)
        nan = torch.zeros_like(out, dtype=torch.bool)
        nan[:, 128:256] = True
        assert torch.equal(out.isnan(), nan)
        nan[:T // 2] = False
        assert torch.equal(two.isnan(), nan)
        assert bool(two[~nan].isfinite().all())


@pytest.mark.parametrize("T,N", [(3, 392), (200, 520), (4100, 4104)])
def test_an_infinite_fp32_weight_scale(mhc, ws, T, N):
    """128 values of k are summed, then scaled: the block's columns are infinite with the sum's sign, the others finite."""
    K = 416
    xq, xs = ref.activations(T, K, 5)
    wq, wsc = ref.weights((), N, K, 6, True)
    wsc[2, 1] = float("inf")
    out = mhc.linear_mxfp8(xq, xs, wq, wsc, out_dtype=torch.float32, workspace=ws)
    mhc.check_status(ws)
    inside = torch.zeros(N, dtype=torch.bool, device="cuda")
    inside[256:384] = True
    assert bool(out[:, ~inside].isfinite().all())
    part = ref.dequant_x(xq, xs)[:, 128:256] @ ref.e4m3_values("cuda")[wq[256:384, 128:256].int()].t()
    sure = part.abs() > 128 * 2.0 ** -23 * (ref.dequant_x(xq, xs)[:, 128:256].abs() @ ref.e4m3_values("cuda")[wq[256:384, 128:256].int()].abs().t())
    got = out[:, inside].double()
    assert bool(sure.any()) and not bool(got.isfinite().any())
    assert torch.equal(got[sure], torch.sign(part[sure]) * math.inf)
