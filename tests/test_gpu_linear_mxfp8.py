"""GPU tests of the 8-bit matrix products (linear_mxfp8, expert_linear_mxfp8) against 64-bit products.

Tolerance per element, from the arithmetic: a product of two E4M3 codes has at most 8 significant bits and the
UE8M0 scales are powers of two, so products are exact in fp32.  K of them are added in fp32 in some order, each
addition off by at most 2^-23 of a partial sum (round to nearest 2^-24; a tensor core may cut off instead), and no
partial sum exceeds S = sum_k |x w|: K 2^-23 S.  fp32 weight scales add a rounding per block of 128, at most
2^-24 S in all.  The fp32 output adds nothing; the bf16 one half a step, 2^-8 of the value."""
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


def check(got, x, w, label=""):
    """got [T, N] against x [T, K] w [N, K]^T (64-bit)."""
    want, S, K = x @ w.t(), x.abs() @ w.abs().t(), x.shape[1]
    tol = K * 2.0 ** -23 * S + 2.0 ** -24 * S
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), f"{label}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


SIZES = [(1, 32, 8), (1, 128, 128), (3, 96, 136), (6, 7168, 1024), (16, 256, 384), (17, 1056, 264), (32, 512, 1000),
         (33, 544, 520), (64, 2048, 256), (65, 288, 136), (128, 1024, 1032), (129, 4064, 328), (300, 1056, 520),
         (513, 2080, 776), (1000, 160, 2056), (2049, 320, 1160),
         (3000, 1056, 7176), (4100, 544, 4104), (5000, 96, 4096),  # the last ones: pairs of CTAs
         (700, 416, 7168), (697, 2080, 7176), (1500, 544, 4096), (1531, 256, 4104)]  # on narrower tiles


@pytest.mark.parametrize("wide", [False, True], ids=["ue8m0", "f32scale"])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_linear_against_64_bits(mhc, ws, T, K, N, wide):
    xq, xs = ref.activations(T, K, T + K, decades=3.0)
    wq, wsc = ref.weights((), N, K, N, wide)
    x, w = ref.dequant_x(xq, xs), ref.dequant_w(wq, wsc)
    f32 = mhc.linear_mxfp8(xq, xs, wq, wsc, out_dtype=torch.float32, workspace=ws)
    bf = mhc.linear_mxfp8(xq.view(torch.float8_e4m3fn), xs, wq.view(torch.float8_e4m3fn), wsc, workspace=ws)
    mhc.check_status(ws)
    assert bf.dtype == torch.bfloat16 and mhc.last_launch_count() == 1
    check(f32, x, w, "fp32")
    check(bf, x, w, "bf16")
    assert torch.equal(bf, f32.bfloat16())  # one accumulation, rounded once


def group(M, E, seed, lo=0, hi=None, empty=()):
    """Random non-decreasing offsets over rows [lo, hi) of M, some experts empty."""
    g = torch.Generator().manual_seed(seed)
    p = torch.rand(E, generator=g) + 0.05
    p[list(empty)] = 0
    hi = M if hi is None else hi
    n = torch.bincount(torch.multinomial(p, hi - lo, replacement=True, generator=g), minlength=E) if hi > lo else torch.zeros(E, dtype=torch.long)
    return torch.cat([torch.tensor([lo]), lo + n.cumsum(0)]).int().cuda()


EXPERTS = [  # M, E, K, N, rows of x (None: no gather)
    (1, 1, 32, 8, None), (1, 8, 128, 128, 3), (12, 8, 512, 264, 6), (48, 64, 1024, 256, 6), (100, 3, 96, 136, None),
    (130, 5, 288, 520, 50), (700, 8, 544, 264, 200), (1500, 16, 416, 392, None), (2000, 2, 1056, 136, 700),
    (77, 1024, 64, 72, 20), (4000, 40, 256, 128, None),
    (6000, 8, 288, 4104, 900), (9000, 40, 160, 2056, None), (3000, 24, 1056, 4096, 700)]  # pairs of CTAs


@pytest.mark.parametrize("wide", [False, True], ids=["ue8m0", "f32scale"])
@pytest.mark.parametrize("M,E,K,N,R", EXPERTS)
def test_expert_linear_against_64_bits(mhc, ws, M, E, K, N, R, wide):
    lo, hi = (0, M) if M < 20 else (3, M - 5)
    off = group(M, E, M + E, lo, hi, empty=range(1, E, 5))
    xq, xs = ref.activations(R or M, K, K, decades=2.0)
    wq, wsc = ref.weights((E,), N, K, N, wide)
    rows = None if R is None else torch.randint(0, R, (M,), generator=torch.Generator().manual_seed(M)).int().cuda()
    x = ref.dequant_x(xq, xs)
    if rows is not None:
        x = x[rows.long()]
    outs = {}
    for dt in (torch.float32, torch.bfloat16):
        out = torch.full((M, N), -7.0, dtype=dt, device="cuda")
        outs[dt] = mhc.expert_linear_mxfp8(xq, xs, wq, wsc, off, rows=rows, out=out, workspace=ws)
        mhc.check_status(ws)
        o = off.tolist()
        assert bool((out[:o[0]] == -7.0).all()) and bool((out[o[-1]:] == -7.0).all())  # left as they were
        for e in range(E):
            if o[e + 1] > o[e]:
                check(out[o[e]:o[e + 1]], x[o[e]:o[e + 1]], ref.dequant_w(wq[e], wsc[e]), f"expert {e}")
    assert torch.equal(outs[torch.float32].bfloat16(), outs[torch.bfloat16])


def test_one_expert_equals_the_plain_product(mhc, ws):
    M, K, N = 150, 672, 392
    xq, xs = ref.activations(M, K, 1)
    wq, wsc = ref.weights((), N, K, 2, False)
    a = mhc.linear_mxfp8(xq, xs, wq, wsc, out_dtype=torch.float32, workspace=ws)
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    b = mhc.expert_linear_mxfp8(xq, xs, wq[None], wsc[None], off, out_dtype=torch.float32, workspace=ws)
    c = mhc.expert_linear_mxfp8(xq, xs, wq[None], wsc[None], off, rows=torch.arange(M, dtype=torch.int32, device="cuda"),
                                out_dtype=torch.float32, workspace=ws)
    x, w = ref.dequant_x(xq, xs), ref.dequant_w(wq, wsc)
    for got in (a, b, c):
        check(got, x, w)
    assert torch.equal(b, c)


def test_one_expert_equals_the_plain_product_in_pairs(mhc, ws):
    M, K, N = 4100, 288, 4104
    xq, xs = ref.activations(M, K, 1)
    wq, wsc = ref.weights((), N, K, 2, True)
    a = mhc.linear_mxfp8(xq, xs, wq, wsc, workspace=ws)
    off = torch.tensor([0, 0, M, M], dtype=torch.int32, device="cuda")
    w3, s3 = torch.stack([wq * 0, wq, wq * 0]), torch.stack([wsc, wsc, wsc])
    b = mhc.expert_linear_mxfp8(xq, xs, w3, s3, off, workspace=ws)
    c = mhc.expert_linear_mxfp8(xq, xs, w3, s3, off, rows=torch.arange(M, dtype=torch.int32, device="cuda"), workspace=ws)
    check(a, ref.dequant_x(xq, xs), ref.dequant_w(wq, wsc))
    assert torch.equal(a, b) and torch.equal(b, c)


def test_overlapping_groups_stay_inside_the_output(mhc, ws):
    """Offsets that go back and forth (not allowed: groups overlap) make more tiles than the rows do; the call still ends,
    and writes nothing outside out."""
    M, K, N, E = 40, 2048, 136, 16
    xq, xs = ref.activations(M, K, 5)
    wq, wsc = ref.weights((E,), N, K, 6, False)
    buf = torch.full((M + 100, N), -7.0, dtype=torch.float32, device="cuda")
    off = torch.tensor([0, M] * 8 + [0], dtype=torch.int32, device="cuda")
    mhc.expert_linear_mxfp8(xq, xs, wq, wsc, off, out=buf[:M], workspace=ws)
    mhc.check_status(ws)
    assert bool((buf[M:] == -7.0).all())


@pytest.mark.parametrize("K", [128, 2048])
def test_offsets_outside_the_rows_are_clamped(mhc, ws, K):
    """A bound outside [0, M] is clamped, a group that ends before it begins is empty; nothing outside out is written."""
    M, N, E = 70, 136, 4
    xq, xs = ref.activations(M, K, 5)
    wq, wsc = ref.weights((E,), N, K, 6, False)
    x = ref.dequant_x(xq, xs)
    buf = torch.full((M + 200, N), -7.0, dtype=torch.float32, device="cuda")
    out = buf[:M]
    off = torch.tensor([-5, 20, 10, 40, 2 ** 31 - 1], dtype=torch.int32, device="cuda")  # groups [0,20) [] [10,40) [40,70)
    mhc.expert_linear_mxfp8(xq, xs, wq, wsc, off, out=out, workspace=ws)
    mhc.check_status(ws)
    check(out[:10], x[:10], ref.dequant_w(wq[0], wsc[0]))
    check(out[20:40], x[20:40], ref.dequant_w(wq[2], wsc[2]))
    check(out[40:], x[40:], ref.dequant_w(wq[3], wsc[3]))
    assert bool((buf[M:] == -7.0).all())
    out.fill_(-7.0)
    mhc.expert_linear_mxfp8(xq, xs, wq, wsc, torch.zeros(E + 1, dtype=torch.int32, device="cuda"), out=out, workspace=ws)
    mhc.check_status(ws)
    assert bool((buf == -7.0).all())  # every group empty


@pytest.mark.parametrize("M,N", [(9, 136), (200, 136), (6000, 4104)])
def test_a_row_index_outside_x_gives_a_row_of_nan(mhc, ws, M, N):
    R, K, E = 10, 256, 3
    xq, xs = ref.activations(R, K, 5)
    wq, wsc = ref.weights((E,), N, K, 6, False)
    rows = torch.randint(0, R, (M,), generator=torch.Generator().manual_seed(1)).int().cuda()
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    for i, v in ((0, -1), (4, R), (M - 1, 2 ** 31 - 1), (5, -2 ** 31)):
        rows[i], bad[i] = v, True
    off = group(M, E, 3)
    out = mhc.expert_linear_mxfp8(xq, xs, wq, wsc, off, rows=rows, out_dtype=torch.float32, workspace=ws)
    mhc.check_status(ws)
    assert bool(out[bad].isnan().all()) and bool(out[~bad].isfinite().all())


@pytest.mark.parametrize("T,N", [(5, 136), (200, 264), (4100, 4104)])
@pytest.mark.parametrize("wide", [False, True], ids=["ue8m0", "f32scale"])
def test_nan_stays_in_its_row_and_column(mhc, ws, T, N, wide):
    K = 416
    xq, xs = ref.activations(T, K, 5)
    wq, wsc = ref.weights((), N, K, 6, wide)
    xq[1, 40] = 0x7F             # a NaN code of x
    wq[9, 411] = 0xFF            # of w
    xs[ref.scale_index(T, K)[3, 12]] = 255   # a NaN scale
    out = mhc.linear_mxfp8(xq, xs, wq, wsc, out_dtype=torch.float32, workspace=ws)
    mhc.check_status(ws)
    nan = torch.zeros_like(out, dtype=torch.bool)
    nan[[1, 3]] = True
    nan[:, 9] = True
    assert torch.equal(out.isnan(), nan)


def test_extreme_scales(mhc, ws):
    """The smallest and largest finite exponents: products that vanish in fp32, and sums at the top of bf16's range."""
    T, K, N = 4, 128, 128
    xq = torch.full((T, K), 0x38, dtype=torch.uint8, device="cuda")    # 1.0
    wq = torch.full((N, K), 0x38, dtype=torch.uint8, device="cuda")
    s = torch.tensor([[0], [127], [240], [1]], dtype=torch.uint8, device="cuda").expand(T, K // 32)
    for b, want in ((127, [None, 128.0, 128.0 * 2.0 ** 113, None]), (0, [0.0, 128.0 * 2.0 ** -127, 128.0 * 2.0 ** -14, 0.0])):
        wsc = torch.full((1, 1), b, dtype=torch.uint8, device="cuda")
        out = mhc.linear_mxfp8(xq, ref.tile_scales(s.contiguous()), wq, wsc, out_dtype=torch.float32, workspace=ws)
        for t in range(T):
            if want[t] is not None:
                assert bool((out[t] == torch.tensor(want[t], dtype=torch.float32)).all()), (b, t, out[t, 0].item())


def test_results_repeat_and_workspaces_stay_clear(mhc, ws):
    """The same bits in every run, on another stream, and captured and replayed beside another graph that shares the
    workspace."""
    xq, xs = ref.activations(6, 4096, 1)
    wq, wsc = ref.weights((), 1024, 4096, 2, True)   # split over k in clusters
    eq, es = ref.weights((8,), 264, 4096, 3, False)
    off = group(6, 8, 1)
    yq, ys = ref.activations(4100, 288, 1)
    vq, vs = ref.weights((), 4104, 288, 2, False)    # pairs of CTAs
    three = mhc.linear_mxfp8(yq, ys, vq, vs, workspace=ws)
    one = mhc.linear_mxfp8(xq, xs, wq, wsc, workspace=ws)
    two = mhc.expert_linear_mxfp8(xq, xs, eq, es, off, workspace=ws)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [torch.empty_like(one) for _ in range(20)], [torch.empty_like(two) for _ in range(20)]
    for a, b in zip(*outs):  # both streams at once
        mhc.linear_mxfp8(xq, xs, wq, wsc, out=a, workspace=ws, stream=s1)
        c = mhc.linear_mxfp8(yq, ys, vq, vs, workspace=ws, stream=s2)
        mhc.expert_linear_mxfp8(xq, xs, eq, es, off, out=b, workspace=ws, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(c, three)
    assert all(torch.equal(a, one) for a in outs[0]) and all(torch.equal(b, two) for b in outs[1])
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    a, b = torch.empty_like(one), torch.empty_like(two)
    with torch.cuda.graph(ga):
        mhc.linear_mxfp8(xq, xs, wq, wsc, out=a, workspace=ws)
    with torch.cuda.graph(gb):
        mhc.expert_linear_mxfp8(xq, xs, eq, es, off, out=b, workspace=ws)
    for _ in range(3):
        a.zero_(), b.zero_()
        ga.replay(), gb.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, one) and torch.equal(b, two)
    mhc.check_status(ws)
    assert not bool(ws.any())


def test_offsets_are_read_when_the_kernel_runs(mhc, ws):
    """A captured call follows the offsets and the rows that its buffers hold at each replay."""
    M, K, N, E = 40, 256, 136, 5
    xq, xs = ref.activations(M, K, 1)
    wq, wsc = ref.weights((E,), N, K, 2, False)
    x = ref.dequant_x(xq, xs)
    off = group(M, E, 1)
    out = torch.zeros(M, N, dtype=torch.float32, device="cuda")
    g = torch.cuda.CUDAGraph()
    mhc.expert_linear_mxfp8(xq, xs, wq, wsc, off, out=out, workspace=ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        mhc.expert_linear_mxfp8(xq, xs, wq, wsc, off, out=out, workspace=ws)
    for seed in (2, 3):
        off.copy_(group(M, E, seed))
        g.replay()
        o = off.tolist()
        for e in range(E):
            check(out[o[e]:o[e + 1]], x[o[e]:o[e + 1]], ref.dequant_w(wq[e], wsc[e]))


def test_outputs_and_weights_beyond_32_bit_offsets(mhc, ws):
    """A result of more than 2^32 bytes and experts' weights of more than 2^32 codes: the ends are right."""
    T, K, N = 300000, 32, 4096
    xq, xs = ref.activations(T, K, 1)
    wq, wsc = ref.weights((), N, K, 2, False)
    out = mhc.linear_mxfp8(xq, xs, wq, wsc, out_dtype=torch.float32, workspace=ws)
    mhc.check_status(ws)
    w = ref.dequant_w(wq, wsc)
    idx = ref.scale_index(T, K, "cuda")
    for sl in (slice(0, 130), slice(262140, 262160), slice(T - 130, T)):
        x = ref.e4m3_values("cuda")[xq[sl].int()] * ref.pow2(xs[idx[sl]]).repeat_interleave(32, 1)
        check(out[sl], x, w)
    del out
    E, K, N = 40, 32768, 4096
    wq = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    one, wsc = ref.weights((E,), 8, K, 3, False)
    wq[:, -8:] = one
    wsc = wsc.expand(E, N // 128, K // 128).contiguous()
    xq, xs = ref.activations(E, K, 4)
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    out = mhc.expert_linear_mxfp8(xq, xs, wq, wsc, off, out_dtype=torch.float32, workspace=ws)
    mhc.check_status(ws)
    x = ref.dequant_x(xq, xs)
    assert not bool(out[:, :-8].any())
    for e in (0, 15, 16, 31, 32, E - 1):
        check(out[e:e + 1, -8:], x[e:e + 1], ref.dequant_w(one[e], wsc[e]))


def test_no_rows(mhc, ws):
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    out = mhc.linear_mxfp8(z(0, 64), z(0), z(16, 64), z(1, 1), workspace=ws)
    assert out.shape == (0, 16) and mhc.last_launch_count() == 0
    out = mhc.expert_linear_mxfp8(z(0, 64), z(0), z(3, 16, 64), z(3, 1, 1), torch.zeros(4, dtype=torch.int32, device="cuda"), workspace=ws)
    assert out.shape == (0, 16)


def test_refusals_leave_the_output_alone(mhc, ws):
    T, K, N = 5, 64, 16
    xq, xs = ref.activations(T, K, 1)
    wq, wsc = ref.weights((), N, K, 2, False)
    out = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    for kw, msg in (({"out_dtype": torch.float16}, "out"), ({"out_dtype": torch.float32}, "out must be float32"),
                    ({"workspace": ws[:128]}, "workspace has 128 bytes"), ({"workspace": ws.cpu()}, "workspace")):
        with pytest.raises((TypeError, ValueError, mhc.MhcError), match=msg):
            mhc.linear_mxfp8(xq, xs, wq, wsc, **{"out": out, "workspace": ws, **kw})
    for args, msg in (((xq.int(), xs, wq, wsc), "x_fp8"), ((xq, xs[:-1], wq, wsc), "x_scales"), ((xq, xs, wq[:, :32], wsc), "w_fp8"),
                      ((xq, xs, wq, wsc.int()), "w_scales"), ((xq, xs, wq, wsc.expand(2, 1)), "w_scales"),
                      ((xq.t().contiguous().t(), xs, wq, wsc), "x_fp8"), ((xq.cpu(), xs, wq, wsc), "x_fp8|x_scales|w_fp8")):
        with pytest.raises((TypeError, ValueError, RuntimeError), match=msg):
            mhc.linear_mxfp8(*args, out=out, workspace=ws)
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError, match="expert_offsets"):
        mhc.expert_linear_mxfp8(xq, xs, wq[None], wsc[None], off.long(), out=out, workspace=ws)
    with pytest.raises(ValueError, match="expert_offsets"):
        mhc.expert_linear_mxfp8(xq, xs, wq[None], wsc[None], off[:1], out=out, workspace=ws)
    with pytest.raises(mhc.MhcError, match="overlaps an input"):
        both = torch.zeros(T * K, dtype=torch.uint8, device="cuda")
        mhc.linear_mxfp8(both.view(T, K), xs, wq, wsc, out=both[:T * N * 2].view(torch.bfloat16).view(T, N), workspace=ws)
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())
