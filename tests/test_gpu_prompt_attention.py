"""GPU checks of the prompt attention against its 64-bit definition (bounds: _attention.attend)."""
import math

import pytest

torch = pytest.importorskip("torch")

import _attention as ref  # noqa: E402
import _mxfp8 as mx  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mhc(mhc_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return mhc_lib


@pytest.fixture(scope="module")
def ws(mhc):
    return torch.zeros(mhc.prompt_workspace_size(), dtype=torch.uint8, device="cuda")


def cum(v, first=0):
    return torch.tensor([first] + (first + torch.tensor(v).cumsum(0)).tolist(), dtype=torch.int32, device="cuda")


def make(T, H, D, seed, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (gain * torch.randn(T, H, D, generator=g, device="cuda")).bfloat16()


def check(o, q, k, v, qn, kn, scale, mode=0, q0=0, k0=0):
    parts, t, j = [], q0, k0
    for n, L in zip(qn, kn):
        if n:
            out, lse, tol, tol_lse = ref.attend(q[t:t + n], k[j:j + L].double(), v[j:j + L].double(), scale, "bf16")
            if "attn_out" in o:
                ref.check_out(o["attn_out"][t:t + n], out, tol)
            if "lse" in o:
                ref.check_lse(o["lse"][t:t + n], lse, tol_lse)
            parts.append((out, tol))
        t, j = t + n, j + L
    if "attn_fp8" in o:
        ref.check_mx(o["attn_fp8"], o["attn_scales"], torch.cat([p[0] for p in parts]).flatten(1), torch.cat([p[1] for p in parts]).flatten(1), mode)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,Hkv", [(1, 3), (2, 2), (3, 1), (7, 2), (8, 2), (12, 1), (16, 1), (33, 1), (64, 1)])
def test_packed_prompts(mhc, ws, D, G, Hkv):
    """Prompts of every length around the tiles' edges in one call, empty ones among them."""
    n = [1, 2, 0, 15, 16, 17, 18, 19, 31, 36, 37, 63, 64, 65, 0, 100, 127, 128, 129, 130, 255, 256, 257, 300]
    T = sum(n)
    q, k, v = make(T, G * Hkv, D, G), make(T, Hkv, D, G + 1, 1.5), make(T, Hkv, D, G + 2)
    o = mhc.prompt_attention(q, k, v, cum(n), cum(n), want_lse=True, workspace=ws)
    mhc.check_status(ws)
    assert sorted(o) == ["attn_out", "lse"]
    check(o, q, k, v, n, n, D ** -0.5)


@pytest.mark.parametrize("D,G,Hkv", [(128, 4, 2), (64, 7, 1), (128, 1, 2), (64, 16, 2)])
@pytest.mark.parametrize("qn,kn", [([1, 3, 129, 40], [700, 3, 130, 513]), ([300], [2000]), ([5, 0, 260], [1, 40, 128]), ([70, 1, 300], [0, 0, 37])])
def test_chunks_after_a_prefix(mhc, ws, D, G, Hkv, qn, kn):
    """More keys than queries (a prefix before them), and fewer (rows that see nothing: zeros and -inf)."""
    q, k, v = make(sum(qn), G * Hkv, D, 1), make(sum(kn), Hkv, D, 2, 1.5), make(sum(kn), Hkv, D, 3)
    o = mhc.prompt_attention(q, k, v, cum(qn), cum(kn), sm_scale=0.2, want_mxfp8=True, want_lse=True, scale_mode=1, workspace=ws)
    mhc.check_status(ws)
    check(o, q, k, v, qn, kn, 0.2, 1)
    t = 0
    for n, L in zip(qn, kn):
        gone = max(0, n - L)
        assert bool((o["attn_out"][t:t + gone] == 0).all()) and bool((o["lse"][t:t + gone] == -math.inf).all())
        t += n


@pytest.mark.parametrize("D,Hq,Hkv,n", [(128, 8, 1, [3000]), (64, 4, 2, [2500, 1, 4100])])
def test_longer_prompts(mhc, ws, D, Hq, Hkv, n):
    T = sum(n)
    q, k, v = make(T, Hq, D, 1, 2.0), make(T, Hkv, D, 2), make(T, Hkv, D, 3)
    o = mhc.prompt_attention(q, k, v, cum(n), cum(n), want_lse=True, workspace=ws)
    check(o, q, k, v, n, n, D ** -0.5)
    again = mhc.prompt_attention(q, k, v, cum(n), cum(n), want_lse=True, workspace=ws)
    assert torch.equal(o["attn_out"], again["attn_out"]) and torch.equal(o["lse"], again["lse"])


@pytest.mark.parametrize("D", [64, 128])
def test_scores_that_differ_by_hundreds(mhc, ws, D):
    """Maxima that rise from tile to tile, and fall: the running rescale."""
    n = 900
    q, k, v = make(n, 4, D, 1), make(n, 2, D, 2), make(n, 2, D, 3)
    ramp = torch.linspace(-1, 1, n, device="cuda")[:, None, None]
    for sign in (1.0, -1.0):
        q[..., 0], k[..., :1] = 8.0, (sign * 300 * ramp).bfloat16()
        o = mhc.prompt_attention(q, k, v, cum([n]), cum([n]), want_lse=True, sm_scale=0.25, workspace=ws)
        check(o, q, k, v, [n], [n], 0.25)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_is_not_seen_is_not_read_into_the_result(mhc, ws, D, bad):
    """NaN and infinities in the rows between and behind the sequences and in later tokens' k and v."""
    n, Hkv, G = [40, 200, 70], 2, 3
    lead, T = 5, 5 + sum([40, 200, 70]) + 300
    q, k, v = make(T, G * Hkv, D, 1), make(T, Hkv, D, 2), make(T, Hkv, D, 3)
    off = cum(n, lead)
    for x in (q, k, v):
        x[:lead] = bad
        x[lead + sum(n):] = bad
    out = torch.full((T, G * Hkv, D), 4.0, dtype=torch.bfloat16, device="cuda")
    o = mhc.prompt_attention(q, k, v, off, off, out={"attn_out": out}, workspace=ws)
    check(o, q, k, v, n, n, D ** -0.5, q0=lead, k0=lead)
    assert bool((out[:lead] == 4).all()) and bool((out[lead + sum(n):] == 4).all())
    at = lead + 40 + 111                        # a token of the second sequence
    for x in (k, v):
        y = x.clone()
        x[at, 1, 3] = bad
        o = mhc.prompt_attention(q, k, v, off, off, workspace=ws)["attn_out"]
        x.copy_(y)
        mine = mhc.prompt_attention(q, k, v, off, off, workspace=ws)["attn_out"]
        before = torch.ones(T, dtype=torch.bool, device="cuda")
        before[at:lead + 240] = False
        before[:lead], before[lead + sum(n):] = False, False
        # (recomputed rows may round otherwise: held to the bound, not to the bits)
        w, _, tol, _ = ref.attend(q[lead + 40:at], k[lead + 40:at].double(), v[lead + 40:at].double(), D ** -0.5, "bf16")
        ref.check_out(o[lead + 40:at], w, tol)
        assert torch.equal(o[lead:lead + 40], mine[lead:lead + 40]) and torch.equal(o[lead + 240:lead + 310], mine[lead + 240:lead + 310])
        assert torch.equal(o[before][:, :G], mine[before][:, :G])   # the other head's
        hit = o[at:lead + 240, G:]
        if x is v:
            assert bool((~hit[..., 3].isfinite()).all()) and bool(hit[..., 4:].isfinite().all())
        elif math.isnan(bad):
            assert bool(hit.isnan().all())


def test_masks_of_the_types_lowest_value(mhc, ws):
    """Scores of -inf and of fp32's lowest: a row whose scores are all -inf is NaN, as 0 / 0 is; beside finite scores they weigh nothing."""
    D, n = 64, 150
    q, k, v = torch.zeros(n, 2, D, device="cuda").bfloat16(), torch.zeros(n, 1, D, device="cuda").bfloat16(), make(n, 1, D, 1)
    q[..., 0] = 1.0
    k[:100, 0, 0] = -math.inf
    o = mhc.prompt_attention(q, k, v, cum([n]), cum([n]), workspace=ws)["attn_out"]
    assert bool(o[:100].isnan().all())
    want, _, tol, _ = ref.attend(q[100:], k[100:].double(), v[100:].double(), 0.125, "bf16")
    ref.check_out(o[100:], want, tol)
    k[:100, 0, 0] = -3.0e38
    q[..., 0] = 8.0                             # products of -2.4e39: -inf in fp32
    o = mhc.prompt_attention(q, k, v, cum([n]), cum([n]), workspace=ws)["attn_out"]
    ref.check_out(o[100:], want, tol)
    q[..., 0] = 1.0
    o = mhc.prompt_attention(q, k, v, cum([n]), cum([n]), workspace=ws)["attn_out"]
    mean, _, tol0, _ = ref.attend(q[:100] * 0, k[:100].double() * 0, v[:100].double(), 0.125, "bf16")
    ref.check_out(o[:100], mean, tol0)          # equal scores, however low
    ref.check_out(o[100:], want, tol)


def test_strided_rows_streams_and_replay(mhc, ws):
    """q, k and v as parts of one product's rows; on another stream; captured and replayed with other offsets."""
    D, Hkv, G, T = 128, 2, 4, 500
    qkv = make(T, G * Hkv + 2 * Hkv, D, 1)
    q, k, v = qkv[:, :G * Hkv], qkv[:, G * Hkv:G * Hkv + Hkv], qkv[:, G * Hkv + Hkv:]
    off = cum([123, 377])
    want = mhc.prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), off, off, want_lse=True, workspace=ws)
    check(want, q, k, v, [123, 377], [123, 377], D ** -0.5)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    o = mhc.prompt_attention(q, k, v, off, off, want_lse=True, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(o["attn_out"], want["attn_out"]) and torch.equal(o["lse"], want["lse"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = mhc.prompt_attention(q, k, v, off, off, want_mxfp8=True, workspace=ws)
    for n in ([123, 377], [500, 0], [1, 499], [250, 250]):
        off.copy_(cum(n))
        graph.replay()
        torch.cuda.synchronize()
        w = mhc.prompt_attention(q, k, v, off, off, want_mxfp8=True, workspace=ws)
        assert all(torch.equal(again[x], w[x]) for x in ("attn_out", "attn_fp8"))
        check(again, q, k, v, n, n, D ** -0.5)
    mhc.check_status(ws)


def test_rows_outside_every_sequence_are_left(mhc, ws):
    D, n = 64, [3, 130]
    T = 10 + sum(n) + 200
    q, k, v = make(T, 4, D, 1), make(T, 2, D, 2), make(T, 2, D, 3)
    K = 4 * D
    out = {"attn_out": torch.full((T, 4, D), 5.0, dtype=torch.bfloat16, device="cuda"), "attn_fp8": torch.full((T, K), 9, dtype=torch.uint8, device="cuda"),
           "attn_scales": torch.full((mx.scale_bytes(T, K),), 77, dtype=torch.uint8, device="cuda"), "lse": torch.full((T, 4), 2.5, device="cuda")}
    o = mhc.prompt_attention(q, k, v, cum(n, 10), cum(n, 10), out=out, workspace=ws)
    rows = slice(10, 10 + sum(n))
    idx = mx.scale_index(T, K, "cuda")
    check({"attn_out": o["attn_out"][rows], "lse": o["lse"][rows], "attn_fp8": o["attn_fp8"][rows], "attn_scales": mx.tile_scales(o["attn_scales"][idx][rows])},
          q[rows], k[rows], v[rows], n, n, D ** -0.5)
    outside = torch.ones(T, dtype=torch.bool, device="cuda")
    outside[rows] = False
    assert bool((o["attn_out"][outside] == 5).all()) and bool((o["attn_fp8"][outside] == 9).all()) and bool((o["lse"][outside] == 2.5).all())
    mask = torch.ones_like(o["attn_scales"], dtype=torch.bool)
    mask[idx[rows].reshape(-1)] = False
    assert bool((o["attn_scales"][mask] == 77).all())


def test_many_short_prompts(mhc, ws):
    n = [(i * 5) % 9 for i in range(1500)]
    T = sum(n)
    q, k, v = make(T, 2, 64, 1), make(T, 1, 64, 2), make(T, 1, 64, 3)
    o = mhc.prompt_attention(q, k, v, cum(n), cum(n), want_lse=True, workspace=ws)
    check(o, q, k, v, n, n, 0.125)


def test_no_keys_at_all(mhc, ws):
    q = make(40, 4, 64, 1)
    k = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    o = mhc.prompt_attention(q, k, k, cum([3, 37]), cum([0, 0]), want_lse=True, want_mxfp8=True, workspace=ws)
    assert bool((o["attn_out"] == 0).all()) and bool((o["lse"] == -math.inf).all()) and bool((o["attn_fp8"] == 0).all())
    mhc.check_status(ws)


@pytest.mark.parametrize("D", [64, 128])
def test_a_query_that_is_not_finite(mhc, ws, D):
    """It makes its own row NaN, and no other."""
    n = [200, 31]
    q, k, v = make(231, 6, D, 1), make(231, 2, D, 2), make(231, 2, D, 3)
    want = mhc.prompt_attention(q, k, v, cum(n), cum(n), workspace=ws)["attn_out"]
    q[100, 4, 9], q[205, 0, 1] = math.nan, -math.inf
    o = mhc.prompt_attention(q, k, v, cum(n), cum(n), workspace=ws)["attn_out"]
    bad = torch.zeros(231, 6, dtype=torch.bool, device="cuda")
    bad[100, 4], bad[205, 0] = True, True
    assert bool(o[bad].isnan().all()) and bool(o[~bad].isfinite().all())
    assert torch.equal(o[~bad], want[~bad])


def test_more_sequences_than_rows(mhc, ws):
    """Empty sequences before, between and behind the others, many more than there are rows."""
    n = [0] * 700 + [1] + [0] * 90 + [5] + [0] * 1100
    q, k, v = make(6, 4, 64, 1), make(6, 4, 64, 2), make(6, 4, 64, 3)
    o = mhc.prompt_attention(q, k, v, cum(n), cum(n), want_lse=True, workspace=ws)
    check(o, q, k, v, n, n, 0.125)


def test_rows_that_take_the_plain_way_over_many_keys(mhc, ws):
    """A value that is not finite behind 20,000 others: its tile's rows are computed plainly, the waits hold."""
    L = 20000
    q, k, v = make(70, 8, 128, 1), make(L, 1, 128, 2), make(L, 1, 128, 3)
    v[L - 1] = math.inf
    o = mhc.prompt_attention(q, k, v, cum([70]), cum([L]), workspace=ws)["attn_out"]
    mhc.check_status(ws)
    want, _, tol, _ = ref.attend(q[:69], k[:L - 1].double(), v[:L - 1].double(), 128 ** -0.5, "bf16")
    ref.check_out(o[:69], want, tol)
    assert bool((~o[69].isfinite()).all())
