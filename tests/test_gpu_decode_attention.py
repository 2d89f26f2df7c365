"""GPU checks of the attention over the 4-bit cache against its 64-bit definition (bounds: _attention.attend)."""
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
    """One workspace for every call, as a program keeps it."""
    return torch.zeros(mhc.decode_workspace_size(), dtype=torch.uint8, device="cuda")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def queries(T, Hq, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed + 77)
    return torch.randn(T, Hq, D, generator=g, device="cuda").bfloat16()


def check(o, b, q, scale, mode=0):
    t = 0
    for i, n in enumerate(b.new):
        if n == 0:
            continue
        out, lse, tol, tol_lse = ref.attend(q[t:t + n], b.k[i], b.v[i], scale, "f16")
        if "attn_out" in o:
            ref.check_out(o["attn_out"][t:t + n], out, tol)
        if "lse" in o:
            ref.check_lse(o["lse"][t:t + n], lse, tol_lse)
        t += n
    if "attn_fp8" in o:
        parts = [ref.attend(q[s:e], b.k[i], b.v[i], scale, "f16") for i, (s, e) in enumerate(zip(b.offsets.tolist(), b.offsets.tolist()[1:])) if e > s]
        ref.check_mx(o["attn_fp8"], o["attn_scales"], torch.cat([p[0] for p in parts]).flatten(1), torch.cat([p[2] for p in parts]).flatten(1), mode)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,Hkv", [(1, 2), (2, 1), (3, 2), (7, 3), (8, 2), (12, 1), (16, 2), (33, 1), (64, 1)])
def test_lengths_and_groups(mhc, ws, D, G, Hkv):
    """One token of each of many sequences, of every length around the tiles' and pages' edges."""
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 100, 127, 128, 129, 255, 257, 400, 513, 1023, 1500]
    b = ref.Batch(mhc, lens, [1] * len(lens), Hkv, D, 16 if D == 64 else 32, seed=G)
    q = queries(b.T, G * Hkv, D, G)
    o = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, want_lse=True, workspace=ws)
    mhc.check_status(ws)
    assert sorted(o) == ["attn_out", "lse"]
    check(o, b, q, D ** -0.5)


@pytest.mark.parametrize("page", [16, 64, 128, 256])
@pytest.mark.parametrize("D,G,Hkv,new", [(128, 8, 2, [6, 1, 0, 2, 6, 4]), (64, 7, 2, [6, 6, 6, 6, 6, 6]), (128, 1, 4, [3, 17, 1, 40, 2, 70]), (64, 16, 1, [5, 1, 9, 0, 3, 33])])
def test_several_tokens_see_their_own(mhc, ws, page, D, G, Hkv, new):
    """Verify blocks: each token sees itself and what is before it.  Also rows of no length, and tokens at positions
    below 0 (they see nothing: zeros and -inf)."""
    lens = [900, 64, 31, 2, 4, 1300]          # the fourth and fifth may be shorter than what is asked of them
    b = ref.Batch(mhc, lens, new, Hkv, D, page, seed=page)
    q = queries(b.T, G * Hkv, D, page)
    o = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, want_mxfp8=True, want_lse=True,
                                   scale_mode=page == 64, sm_scale=0.11, workspace=ws)
    mhc.check_status(ws)
    check(o, b, q, 0.11, int(page == 64))
    t = b.offsets.tolist()
    for i, n in enumerate(new):
        gone = max(0, n - lens[i])
        assert bool((o["attn_out"][t[i]:t[i] + gone] == 0).all()) and bool((o["lse"][t[i]:t[i] + gone] == -math.inf).all())


@pytest.mark.parametrize("D,Hkv,G,lens", [(128, 1, 8, [40000]), (64, 2, 4, [70001, 5]), (128, 2, 3, [20000, 1, 9000, 0, 12345])])
def test_long_sequences_are_split_and_joined(mhc, ws, D, Hkv, G, lens):
    b = ref.Batch(mhc, lens, [1] * len(lens), Hkv, D, 64, seed=D)
    q = queries(b.T, G * Hkv, D, 3) * 2
    o = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, want_lse=True, workspace=ws)
    check(o, b, q, D ** -0.5)
    again = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, want_lse=True, workspace=ws)
    assert torch.equal(o["attn_out"], again["attn_out"]) and torch.equal(o["lse"], again["lse"])
    mhc.check_status(ws)


def test_many_rows_and_cut_sequences(mhc, ws):
    """More rows than eight warps each are joined by, most of their sequences cut."""
    lens = [2000 + 37 * i for i in range(40)]
    b = ref.Batch(mhc, lens, [1] * 40, 8, 64, 64, seed=12)
    q = queries(b.T, 32, 64, 12)
    o = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, want_lse=True, want_mxfp8=True, workspace=ws)
    check(o, b, q, 0.125)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("spread,qs", [(6.0, 1.0), (0.0, 40.0), (0.0, 2.0 ** -30), (12.0, 2.0 ** -20)])
def test_scales_and_queries_of_every_magnitude(mhc, ws, D, spread, qs):
    """Scales that differ by many powers of two from token to token, scores that differ by hundreds, and tiny queries."""
    b = ref.Batch(mhc, [700, 33, 260], [2, 1, 4], 2, D, 32, seed=9, spread=spread)
    q = (queries(b.T, 8, D, 5).float() * qs).bfloat16()
    o = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, want_lse=True, workspace=ws)
    check(o, b, q, D ** -0.5)


def test_a_small_v_under_a_large_one_that_is_not_looked_at(mhc, ws):
    """V scales 2^20 apart: where the large V's token has no weight, the small ones' sum keeps its precision."""
    D, L = 128, 300
    b = ref.Batch(mhc, [L], [1], 1, D, 32, seed=1)
    k = torch.zeros(L, 1, D, dtype=torch.float64, device="cuda")
    k[:, 0, 0] = 4.0
    k[137, 0, 0] = -4.0
    v = torch.randn(L, 1, D, dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    v[137] *= 2.0 ** 20
    pos = torch.arange(L, device="cuda")
    for part, x in enumerate((k, v)):
        ref.put(b.cache, b.page_table, 0, pos, part, *ref.quantize4(x, 0))
    b.k, b.v = [[ref.get(b.cache, b.page_table, 0, pos, p)] for p in (0, 1)]
    q = torch.zeros(1, 4, D, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = 6.0                             # scores 24 and -24: 2^-69 of the weight, 2^-49 of the largest V
    o = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, sm_scale=1.0, workspace=ws)
    out, _, tol, _ = ref.attend(q, b.k[0], b.v[0], 1.0, "f16")
    small = (tol - b.v[0].abs().max() * 2.0 ** -36).clamp(min=0) + 2.0 ** -20 * out.abs()   # the bound without the part that the large V has
    ref.check_out(o["attn_out"], out, small + 2.0 ** -24)


@pytest.mark.parametrize("D,G,lens,new,E", [(128, 4, [300, 70, 5], [6, 3, 5], 60), (64, 7, [97, 33, 40000], [40, 2, 6], 24), (128, 1, [64, 31], [64, 9], 100)])
def test_a_later_large_v_leaves_earlier_rows_their_bits(mhc, ws, D, G, lens, new, E):
    """V grows by 2^E from each new token to the next two: a row's result is bounded by the V that it sees itself."""
    b = ref.Batch(mhc, lens, new, 2, D, 16, seed=E)
    for i, (n, m) in enumerate(zip(lens, new)):
        pos = torch.arange(n, device="cuda")
        v = torch.randn(n, 2, D, dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(i))
        up = ((pos - (n - m)).clamp(min=0) // 2 * E).clamp(max=120).double()
        v = v * torch.exp2(up - 20)[:, None, None]
        ref.put(b.cache, b.page_table, i, pos, 1, *ref.quantize4(v, 0))
        b.v[i] = ref.get(b.cache, b.page_table, i, pos, 1)
    q = queries(b.T, G * 2, D, 8)
    o = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, want_lse=True, workspace=ws)
    mhc.check_status(ws)
    t = 0
    for i, (n, m) in enumerate(zip(lens, new)):
        for j in range(m):
            end = n - m + j + 1
            if end > 0:
                out, lse, tol, tol_lse = ref.attend(q[t:t + 1], b.k[i][:end], b.v[i][:end], D ** -0.5, "f16")
                ref.check_out(o["attn_out"][t:t + 1], out, tol)
                ref.check_lse(o["lse"][t:t + 1], lse, tol_lse)
            t += 1


@pytest.mark.parametrize("lens", [[90, 40000], [2000 + 37 * i for i in range(40)]])
def test_the_largest_v_of_cut_sequences(mhc, ws, lens):
    """Magnitudes up to bf16's last binades: neither the parts' sums nor their join leave fp32's range."""
    D, Hkv = 64, 8
    b = ref.Batch(mhc, lens, [1] * len(lens), Hkv, D, 64, seed=13)
    for i, n in enumerate(lens):
        v = torch.rand(n, Hkv, D, dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(i)) * 2.0 ** 127
        pos = torch.arange(n, device="cuda")
        ref.put(b.cache, b.page_table, i, pos, 1, *ref.quantize4(v, 0))
        b.v[i] = ref.get(b.cache, b.page_table, i, pos, 1)
    q = queries(b.T, 32, D, 13)
    o = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, want_lse=True, workspace=ws)
    check(o, b, q, D ** -0.5)


@pytest.mark.parametrize("page", [16, 128])
def test_what_is_not_seen_is_not_read_into_the_result(mhc, ws, page):
    """NaN scales and every code in the rest of a page (Batch fills it with 255), NaN in the later tokens of a block."""
    D, Hkv, G = 128, 2, 4
    b = ref.Batch(mhc, [70, 200], [5, 3], Hkv, D, page, seed=4)
    q = queries(b.T, G * Hkv, D, 6)
    nan = torch.full((1, Hkv, D), math.nan, dtype=torch.float64, device="cuda")
    for part in (0, 1):                         # the third token of the first block
        ref.put(b.cache, b.page_table, 0, torch.tensor([67], device="cuda"), part, *ref.quantize4(nan, 0))
    o = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, want_lse=True, workspace=ws)["attn_out"]
    out, _, tol, _ = ref.attend(q[:2], b.k[0][:67], b.v[0][:67], D ** -0.5, "f16")
    ref.check_out(o[:2], out, tol)
    assert bool(o[2:5].isnan().all())
    out, _, tol, _ = ref.attend(q[5:8], b.k[1], b.v[1], D ** -0.5, "f16")
    ref.check_out(o[5:8], out, tol)
    # NaN in V alone, and in one block of it: that block of the rows that see it
    b = ref.Batch(mhc, [70], [5], Hkv, D, page, seed=4)
    v = b.v[0][67:68].clone()
    v[:, 1, 40] = math.nan
    ref.put(b.cache, b.page_table, 0, torch.tensor([67], device="cuda"), 1, *ref.quantize4(v, 0))
    o = mhc.decode_attention_mxfp4(q[:5], b.cache, b.page_table, b.seq_lens, b.offsets, workspace=ws)["attn_out"]
    hit = torch.zeros(5, G * Hkv, D, dtype=torch.bool, device="cuda")
    hit[2:, G:, 32:64] = True
    assert torch.equal(o.isnan(), hit)


def test_places_that_do_not_exist(mhc, ws):
    """Pages outside the cache and lengths beyond the table give NaN to the rows that see them, and to no other."""
    D, Hkv = 64, 2
    b = ref.Batch(mhc, [40, 100, 64, 80], [4, 2, 3, 2], Hkv, D, 16, seed=8)
    q = queries(b.T, 4, D, 8)
    out, _, tol, _ = ref.attend(q[:4], b.k[0], b.v[0], D ** -0.5, "f16")
    last, _, tol_last, _ = ref.attend(q[9:11], b.k[3], b.v[3], D ** -0.5, "f16")
    b.page_table[1, 2] = b.cache.shape[0]       # one page of the second sequence
    b.page_table[2, 0] = -7
    b.page_table[2, 3] = 2147483647
    o = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, want_lse=True, workspace=ws)
    ref.check_out(o["attn_out"][:4], out, tol)
    ref.check_out(o["attn_out"][9:11], last, tol_last)
    assert bool(o["attn_out"][4:9].isnan().all()) and bool(o["lse"][4:9].isnan().all())
    room = b.page_table.shape[1] * 16
    b.seq_lens.copy_(i32([40, 2147483647, -5, room + 1]))
    o = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, want_lse=True, workspace=ws)
    ref.check_out(o["attn_out"][:4], out, tol)
    assert bool(o["attn_out"][4:6].isnan().all()) and bool(o["attn_out"][10].isnan().all())
    assert bool((o["attn_out"][6:9] == 0).all()) and bool((o["lse"][6:9] == -math.inf).all())


def test_rows_outside_and_strides(mhc, ws):
    """q as a part of a wider row; rows before the first and behind the last sequence are left as they were."""
    D, Hkv, G = 128, 2, 3
    b = ref.Batch(mhc, [50, 333], [2, 3], Hkv, D, 64, seed=2)
    T = 4 + b.T + 140
    wide = queries(T, 11, D, 1)
    q = wide[:, 2:2 + G * Hkv]
    off = b.offsets + 4
    out = {"attn_out": torch.full((T, 6, D), 5.0, dtype=torch.bfloat16, device="cuda"), "attn_fp8": torch.full((T, 6 * D), 9, dtype=torch.uint8, device="cuda"),
           "attn_scales": torch.full((mx.scale_bytes(T, 6 * D),), 77, dtype=torch.uint8, device="cuda"), "lse": torch.full((T, 6), 2.5, device="cuda")}
    o = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, off, out=out, workspace=ws)
    assert all(o[n] is out[n] for n in out)
    rows = slice(4, 4 + b.T)
    idx = mx.scale_index(T, 6 * D, "cuda")
    tiles = mx.tile_scales(o["attn_scales"][idx][rows])
    check({"attn_out": o["attn_out"][rows], "attn_fp8": o["attn_fp8"][rows], "attn_scales": tiles, "lse": o["lse"][rows]}, b, q[rows], D ** -0.5)
    outside = torch.ones(T, dtype=torch.bool, device="cuda")
    outside[rows] = False
    assert bool((o["attn_out"][outside] == 5).all()) and bool((o["attn_fp8"][outside] == 9).all()) and bool((o["lse"][outside] == 2.5).all())
    mask = torch.ones_like(o["attn_scales"], dtype=torch.bool)
    mask[idx[rows].reshape(-1)] = False
    assert bool((o["attn_scales"][mask] == 77).all())


def test_streams_graphs_and_shared_geometry(mhc):
    """Captured and replayed with new lengths, and two workspaces on two streams at once: the results of calls alone."""
    D, Hkv, G = 128, 2, 8
    b = ref.Batch(mhc, [5000, 900, 40], [1, 1, 1], Hkv, D, 64, seed=5)
    q = queries(b.T, G * Hkv, D, 2)
    w = [torch.zeros(mhc.decode_workspace_size(), dtype=torch.uint8, device="cuda") for _ in range(2)]
    call = lambda x, ws, **k: mhc.decode_attention_mxfp4(x, b.cache, b.page_table, b.seq_lens, b.offsets, workspace=ws, **k)["attn_out"]  # noqa: E731
    want, want2 = call(q, w[0]), call(-q, w[0])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got.append(call(q, w[0], stream=streams[0]))
        got.append(call(-q, w[1], stream=streams[1]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, (want, want2)[i % 2]) for i, x in enumerate(got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(q, w[0])
    for lens in ([5000, 900, 40], [1, 17, 2], [4999, 0, 33]):
        b.seq_lens.copy_(i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call(q, w[1]))
    mhc.check_status(w[0])


def test_more_sequences_than_threads(mhc, ws):
    B = 1100
    lens = [(b * 7) % 40 for b in range(B)]
    b = ref.Batch(mhc, lens, [1 + (i % 3 == 0) for i in range(B)], 1, 64, 16, seed=6)
    q = queries(b.T, 2, 64, 4)
    o = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, want_lse=True, workspace=ws)
    check(o, b, q, 0.125)


@pytest.mark.parametrize("E", [-126, -124, -100, 100])
def test_values_at_the_ends_of_the_range(mhc, ws, E):
    """V of the smallest scales, fp32's subnormals among the results, and large ones."""
    D = 64
    b = ref.Batch(mhc, [90, 40000], [1, 1], 1, D, 32, seed=3)
    for i, n in enumerate(b.lens):
        v = torch.randn(n, 1, D, dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(i)) * 2.0 ** E
        pos = torch.arange(n, device="cuda")
        ref.put(b.cache, b.page_table, i, pos, 1, *ref.quantize4(v, 0))
        b.v[i] = ref.get(b.cache, b.page_table, i, pos, 1)
    q = queries(2, 4, D, 4)
    o = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, workspace=ws)["attn_out"]
    for i in range(2):
        out, _, tol, _ = ref.attend(q[i:i + 1], b.k[i], b.v[i], D ** -0.5, "f16")
        ref.check_out(o[i:i + 1], out, tol)
        assert float(o[i].abs().amax()) > 0


@pytest.mark.parametrize("n,Hq", [(1, 4), (6, 14)])
def test_a_query_that_is_not_finite(mhc, ws, n, Hq):
    """It makes its own rows NaN, and no other."""
    D = 128
    b = ref.Batch(mhc, [300, 70], [n, n], 2, D, 32, seed=3)
    q = queries(b.T, Hq, D, 4)
    want = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, workspace=ws)["attn_out"]
    q[0, 1, 5], q[n, Hq - 1, 7] = math.nan, math.inf
    o = mhc.decode_attention_mxfp4(q, b.cache, b.page_table, b.seq_lens, b.offsets, workspace=ws)["attn_out"]
    bad = torch.zeros(b.T, Hq, dtype=torch.bool, device="cuda")
    bad[0, 1], bad[n, Hq - 1] = True, True
    assert bool(o[bad].isnan().all())
    for i in range(2):   # (a rescale at another time may round otherwise: held to the bound)
        out, _, tol, _ = ref.attend(q[i * n:i * n + n].nan_to_num(0, 0, 0), b.k[i], b.v[i], D ** -0.5, "f16")
        keep = ~bad[i * n:i * n + n]
        ref.check_out(o[i * n:i * n + n][keep], out[keep], tol[keep])
    assert bool(want.isfinite().all())
