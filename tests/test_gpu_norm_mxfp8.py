"""GPU tests of the MXFP8 producers (add_rmsnorm_mxfp8, swiglu_mxfp8) against their 64-bit definitions.

Tolerances, from the arithmetic:
  * residual_out = bf16(x + residual): one fp32 addition, then the bf16 rounding: 2^-8 (1 + 2^-16) of the value.
  * layer_in: one bf16 rounding (2^-8) of a value that is off by less than 2^-20 before it.  The square sum, of terms of
    one sign: 5 roundings within a vector of 8 (product, three fused additions, the two halves), one addition per
    vector of a thread (at most 16, H = 65536), twice 5 in the sums over lanes: 31 of 2^-24, halved by the root; the
    root as a pair, and two roundings.  Asked: 2^-8 + 2^-19.
  * codes and scale bytes of the norm: those of the kernel's own bf16 layer input, bit for bit.
  * codes of the SwiGLU: the correctly rounded code of the exact value wherever that is a normal E4M3 number; below
    (|value| < 2^-6 after scaling) fp32's error may move a value across a border: one step, 2^-9, at most; the scale
    bytes are exact."""
import pytest

torch = pytest.importorskip("torch")

import _mxfp8 as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mhc(mhc_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return mhc_lib


def check_mx(codes, tiles, y, block, mode, exact_subnormals=True):
    """codes and scale tiles against the quantization of y (64-bit values); returns nothing, asserts."""
    M, K = y.shape
    want, E = ref.quantize(y, block, mode)
    got_e = tiles[ref.scale_index(M, K, codes.device)].int() - 127
    assert torch.equal(got_e, E), f"{int((got_e != E).sum())} scale bytes differ"
    got = ref.e4m3_values(codes.device)[codes.int()]
    off = (got - want).abs()
    ok = off == 0 if exact_subnormals else (off == 0) | ((want.abs() <= 2.0 ** -6) & (off <= 2.0 ** -9))
    assert bool(ok.all()), f"{int((~ok).sum())} codes differ"


def norm_inputs(T, H, seed, residual=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    scale = 10.0 ** (4 * torch.rand(T, 1, generator=g, device="cuda") - 2)
    x = (torch.randn(T, H, generator=g, device="cuda") * scale).bfloat16()
    r = (3 * torch.randn(T, H, generator=g, device="cuda") * scale).bfloat16() if residual else None
    w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).bfloat16()
    return x, r, w


def norm_ref(s, w, eps):
    v = s.double()
    return v / (v.square().mean(1, keepdim=True) + eps).sqrt() * w.double()


@pytest.mark.parametrize("block,mode", [(32, 0), (32, 1), (128, 0), (128, 1)])
@pytest.mark.parametrize("T,H", [(1, 32), (1, 7168), (3, 96), (6, 1024), (7, 2048), (130, 2080), (33, 4096), (5, 4128),
                                 (257, 7168), (2, 8192), (9, 8224), (3, 16384), (2, 65536)])
def test_add_rmsnorm_against_64_bits(mhc, T, H, block, mode):
    x, r, w = norm_inputs(T, H, T + H)
    eps = 2e-6
    o = mhc.add_rmsnorm_mxfp8(x, r, w, rmsnorm_eps=eps, scale_mode=mode, scale_block=block, want_bf16=True)
    assert mhc.last_launch_count() == 1
    s = x.double() + r.double()
    assert bool(((o["residual_out"].double() - s).abs() <= 2.0 ** -8 * (1 + 2.0 ** -16) * s.abs()).all())
    y = norm_ref(o["residual_out"], w, eps)
    assert bool(((o["layer_in"].double() - y).abs() <= (2.0 ** -8 + 2.0 ** -19) * y.abs() + 2.0 ** -133).all())
    check_mx(o["layer_in_fp8"], o["layer_in_scales"], o["layer_in"].double(), block, mode)
    # the other forms give the same bits: without the bf16 output, only the bf16 output, without the residual's output
    a = mhc.add_rmsnorm_mxfp8(x, r, w, rmsnorm_eps=eps, scale_mode=mode, scale_block=block)
    b = mhc.add_rmsnorm_mxfp8(x, r, w, rmsnorm_eps=eps, want_bf16=True, want_mxfp8=False)
    c = mhc.add_rmsnorm_mxfp8(x, r, w, rmsnorm_eps=eps, scale_mode=mode, scale_block=block, out={"residual_out": None})
    d = mhc.add_rmsnorm_mxfp8(o["residual_out"], None, w, rmsnorm_eps=eps, scale_mode=mode, scale_block=block)
    idx = ref.scale_index(T, H, "cuda")
    for q in (a, c, d):
        assert torch.equal(q["layer_in_fp8"], o["layer_in_fp8"])
        assert torch.equal(q["layer_in_scales"][idx], o["layer_in_scales"][idx])
    assert torch.equal(a["residual_out"], o["residual_out"]) and torch.equal(b["layer_in"], o["layer_in"])
    assert "layer_in" not in a and "layer_in_fp8" not in b and "residual_out" not in d


def test_bf16_only_takes_any_row_of_whole_vectors(mhc):
    for H in (8, 24, 1000, 4104):
        x, r, w = norm_inputs(3, H, H)
        o = mhc.add_rmsnorm_mxfp8(x, r, w, rmsnorm_eps=1e-5, want_bf16=True, want_mxfp8=False)
        y = norm_ref(o["residual_out"], w, 1e-5)
        assert bool(((o["layer_in"].double() - y).abs() <= (2.0 ** -8 + 2.0 ** -19) * y.abs() + 2.0 ** -133).all())


@pytest.mark.parametrize("H", [1024, 8224])
def test_residual_in_place_padding_untouched_and_special_rows(mhc, H):
    """The residual updated in place; the scale tiles' padding bytes stay; a row of zeros gives zero codes with the
    smallest exponent; NaN and infinity stay in their rows."""
    T = 6
    x, r, w = norm_inputs(T, H, 9)
    x[1], r[1] = 0, 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    want = mhc.add_rmsnorm_mxfp8(x, r, w, rmsnorm_eps=2e-6)
    tiles = torch.full((mhc.mxfp8_scale_bytes(T, H),), 0xA5, dtype=torch.uint8, device="cuda")
    o = mhc.add_rmsnorm_mxfp8(x, r, w, rmsnorm_eps=2e-6, out={"residual_out": r, "layer_in_scales": tiles})
    assert o["residual_out"] is r
    assert torch.equal(r.view(torch.int16), want["residual_out"].view(torch.int16))
    assert torch.equal(o["layer_in_fp8"], want["layer_in_fp8"])
    idx = ref.scale_index(T, H, "cuda")
    pad = torch.ones_like(tiles, dtype=torch.bool)
    pad[idx.reshape(-1)] = False
    assert bool((tiles[pad] == 0xA5).all())
    v = ref.e4m3_values("cuda")[o["layer_in_fp8"].int()]
    assert not bool(v[1].any()) and not bool(tiles[idx[1]].any())
    assert bool(v[2].isnan().all())                      # a NaN makes the whole norm NaN
    assert bool(v[3, 7].isnan()) and not bool(v[3, :7].any()) and not bool(v[3, 8:].any())  # inf/inf, x/inf
    assert bool(v[[0, 4, 5]].isfinite().all())


@pytest.mark.parametrize("T,H", [(9001, 512), (5003, 992), (3001, 2048), (1501, 4096), (1003, 7168), (1201, 8192), (700, 8224)])
def test_rows_in_turn(mhc, T, H):
    """More rows than run at once: those of the formula, and the bits of calls of a few rows, the residual in place or not;
    NaN and infinity stay in their rows."""
    x, r, w = norm_inputs(T, H, T)
    x[T // 2, 3] = float("nan")
    x[T // 3, H - 1] = float("inf")
    o = mhc.add_rmsnorm_mxfp8(x, r, w, rmsnorm_eps=2e-6, want_bf16=True)
    mild = torch.ones(T, dtype=torch.bool, device="cuda")
    mild[[T // 2, T // 3]] = False
    y = norm_ref(o["residual_out"][mild], w, 2e-6)
    assert bool(((o["layer_in"][mild].double() - y).abs() <= (2.0 ** -8 + 2.0 ** -19) * y.abs() + 2.0 ** -133).all())
    assert bool(o["layer_in"][T // 2].isnan().all()) and not bool(o["layer_in"][mild].isnan().any())
    idx = ref.scale_index(T, H, "cuda")
    for lo in (0, T // 2 - 50, T - 100):
        few = mhc.add_rmsnorm_mxfp8(x[lo:lo + 100].clone(), r[lo:lo + 100].clone(), w, rmsnorm_eps=2e-6, want_bf16=True)
        for k in ("residual_out", "layer_in"):
            assert torch.equal(few[k].view(torch.int16), o[k][lo:lo + 100].view(torch.int16))
        assert torch.equal(few["layer_in_fp8"], o["layer_in_fp8"][lo:lo + 100])
        assert torch.equal(few["layer_in_scales"][ref.scale_index(100, H, "cuda")], o["layer_in_scales"][idx[lo:lo + 100]])
    again = mhc.add_rmsnorm_mxfp8(x, r, w, rmsnorm_eps=2e-6, out={"residual_out": r})
    assert torch.equal(r.view(torch.int16), o["residual_out"].view(torch.int16))
    assert torch.equal(again["layer_in_fp8"], o["layer_in_fp8"])
    assert torch.equal(again["layer_in_scales"][idx], o["layer_in_scales"][idx])


@pytest.mark.parametrize("block,mode", [(32, 0), (32, 1), (128, 0), (128, 1)])
@pytest.mark.parametrize("T,F", [(1, 32), (1, 2048), (3, 96), (48, 2048), (130, 160), (77, 1056), (1000, 512), (2, 65536),
                                 (5000, 544), (4097, 2048)])  # several rounds
def test_swiglu_against_64_bits(mhc, T, F, block, mode):
    g = torch.Generator(device="cuda").manual_seed(T + F)
    gu = (torch.randn(T, 2 * F, generator=g, device="cuda") * 10.0 ** (2 * torch.rand(T, 1, generator=g, device="cuda") - 1)).bfloat16()
    tiles = torch.full((mhc.mxfp8_scale_bytes(T, F),), 0xA5, dtype=torch.uint8, device="cuda")
    o = mhc.swiglu_mxfp8(gu, scale_mode=mode, scale_block=block, out={"act_scales": tiles})
    assert mhc.last_launch_count() == 1
    a, b = gu[:, :F].double(), gu[:, F:].double()
    check_mx(o["act_fp8"], tiles, a / (1 + torch.exp(-a)) * b, block, mode, exact_subnormals=False)
    pad = torch.ones_like(tiles, dtype=torch.bool)
    pad[ref.scale_index(T, F, "cuda").reshape(-1)] = False
    assert bool((tiles[pad] == 0xA5).all())


def test_swiglu_extreme_values(mhc):
    """Gates where the exponential overflows or vanishes, zeros, NaN and infinities: in 64 bits the same."""
    F = 64
    gate = torch.tensor([-1e38, -200.0, -100.0, -88.5, -30.0, -1e-3, -0.0, 0.0, 1e-30, 1e-3, 1.0, 30.0, 100.0, 1e30, 3e38, 5.0]).repeat(4)
    up = torch.tensor([1.0, -2.0, 1e4, 1e-8]).repeat_interleave(16)
    gu = torch.cat([gate, up])[None].repeat(5, 1)
    gu[1, 3], gu[2, F + 40], gu[3, 20] = float("nan"), float("nan"), float("-inf")
    gu[4] = 0
    gu = gu.bfloat16().cuda()
    o = mhc.swiglu_mxfp8(gu)
    v = ref.e4m3_values("cuda")[o["act_fp8"].int()]
    a, b = gu[:1, :F].double(), gu[:1, F:].double()
    check_mx(o["act_fp8"][:1], o["act_scales"], a / (1 + torch.exp(-a)) * b, 32, 0, exact_subnormals=False)
    nan = torch.zeros(4, F, dtype=torch.bool)
    nan[1, 3] = nan[2, 40] = nan[3, 20] = True   # -inf: -inf / (1 + inf)
    assert torch.equal(v[:4].isnan().cpu(), nan)
    assert not bool(v[4].any())


def test_captured_and_on_another_stream(mhc):
    x, r, w = norm_inputs(40, 1024, 3)
    gu = torch.randn(40, 2048, device="cuda").bfloat16()
    want = mhc.add_rmsnorm_mxfp8(x, r, w, rmsnorm_eps=2e-6)
    act = mhc.swiglu_mxfp8(gu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o1, o2 = mhc.add_rmsnorm_mxfp8(x, r, w, rmsnorm_eps=2e-6, stream=s), mhc.swiglu_mxfp8(gu, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o3, o4 = mhc.add_rmsnorm_mxfp8(x, r, w, rmsnorm_eps=2e-6), mhc.swiglu_mxfp8(gu)
    g.replay()
    torch.cuda.synchronize()
    for o in (o1, o3):
        assert all(torch.equal(o[k], want[k]) for k in ("residual_out", "layer_in_fp8"))
    for o in (o2, o4):
        assert torch.equal(o["act_fp8"], act["act_fp8"])


def test_no_tokens_and_refusals(mhc):
    x, r, w = norm_inputs(4, 64, 1)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    assert mhc.add_rmsnorm_mxfp8(e, e, w, rmsnorm_eps=1e-6)["layer_in_fp8"].shape == (0, 64)
    assert mhc.swiglu_mxfp8(e)["act_fp8"].shape == (0, 32)
    for kw, msg in (({"scale_block": 64}, "scale_block"), ({"scale_mode": 2}, "scale mode"), ({"rmsnorm_eps": float("nan")}, "rmsnorm_eps")):
        with pytest.raises(mhc.MhcError, match=msg):
            mhc.add_rmsnorm_mxfp8(x, r, w, **{"rmsnorm_eps": 1e-6, **kw})
    with pytest.raises(mhc.MhcError, match="multiple of 32"):
        mhc.add_rmsnorm_mxfp8(x[:, :40].contiguous(), None, w[:40].contiguous(), rmsnorm_eps=1e-6,
                              out={"layer_in_scales": torch.zeros(0, dtype=torch.uint8, device="cuda")})
    with pytest.raises(mhc.MhcError, match="are NULL"):
        mhc.add_rmsnorm_mxfp8(x, r, w, rmsnorm_eps=1e-6, want_mxfp8=False)
    with pytest.raises(mhc.MhcError, match="overlaps an input"):
        mhc.add_rmsnorm_mxfp8(x, r, w, rmsnorm_eps=1e-6, out={"residual_out": x})
    with pytest.raises(ValueError, match="residual has shape"):
        mhc.add_rmsnorm_mxfp8(x, r[:2], w, rmsnorm_eps=1e-6)
    with pytest.raises(TypeError, match="gate_up must be bfloat16"):
        mhc.swiglu_mxfp8(x.float())
    with pytest.raises(mhc.MhcError, match="multiple of 32"):
        mhc.swiglu_mxfp8(x[:, :16].contiguous(), out={"act_scales": torch.zeros(0, dtype=torch.uint8, device="cuda")})
