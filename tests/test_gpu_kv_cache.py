"""GPU checks of the 4-bit cache: what is written and read back, byte for byte against the format's definition."""
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


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def table(lens, page, seed=0):
    need = [-(-n // page) for n in lens]
    P, W = sum(need) + 2, max(max(need), 1)
    order = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).int()
    t = torch.full((len(lens), W), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t.cuda(), P


def cum(v):
    return i32([0] + torch.tensor(v).cumsum(0).tolist())


def special(T, H, D, dtype, seed):
    """Values of every magnitude, with blocks of zeros, ties, subnormals, infinities and NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, D // 32, 32, generator=g, device="cuda")
    x = x * torch.exp2(torch.randint(-130, 120, (T, H, D // 32, 1), generator=g, device="cuda").float())
    kind = torch.randint(0, 12, (T, H, D // 32), generator=g, device="cuda")
    grid = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 7.999, 0.2, -0.25, -5, -0.1, 0.0, -0.0], device="cuda")
    ties = grid[torch.randint(0, 16, x.shape, generator=g, device="cuda")]
    ties[..., 0] = torch.where(ties[..., 0] < 4, 4.0, ties[..., 0])
    x = torch.where((kind == 0)[..., None], torch.zeros_like(x), x)
    x = torch.where((kind == 1)[..., None], -torch.zeros_like(x), x)
    x = torch.where((kind == 2)[..., None], ties * 2.0 ** 5, x)
    x = torch.where((kind == 3)[..., None], ties, x)
    x = torch.where((kind == 4)[..., None], x.clamp(-1, 1) * 2.0 ** -126, x)
    x[..., 5] = torch.where(kind == 5, math.inf, x[..., 5])
    x[..., 7] = torch.where(kind == 6, -math.inf, x[..., 7])
    x[..., 9] = torch.where(kind == 7, math.nan, x[..., 9])
    return x.reshape(T, H, D).to(dtype)


@pytest.mark.parametrize("D,Hkv,page", [(128, 1, 16), (128, 3, 64), (64, 2, 32), (64, 8, 128), (128, 8, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mode", [0, 1])
def test_write_is_the_definition(mhc, D, Hkv, page, dtype, mode):
    new, before = [1, 0, 17, 64, 130, 5], [0, 9, 15, 1, 200, 31]
    lens = [n + p for n, p in zip(new, before)]
    pt, P = table(lens, page)
    T = sum(new)
    qkv = special(T + 3, 3 * Hkv, D, dtype, 5 + mode).view(T + 3, 3, Hkv, D)   # rows behind the last sequence, and parts of wider rows
    k, v = qkv[:, 1], qkv[:, 2]
    want = torch.randint(0, 256, mhc.kv_cache_shape(P, Hkv, page, D), generator=torch.Generator("cuda").manual_seed(1), device="cuda", dtype=torch.uint8)
    cache = want.clone()
    assert mhc.kv_write_mxfp4(k, v, cache, pt, i32(lens), cum(new), scale_mode=mode) is cache
    t = 0
    for b, n in enumerate(new):
        pos = torch.arange(before[b], lens[b], device="cuda")
        for part, x in enumerate((k, v)):
            ref.put(want, pt, b, pos, part, *ref.quantize4(x[t:t + n].double(), mode))
        t += n
    assert torch.equal(cache, want)
    # and back: exact in bf16 but where a value leaves its range
    o = mhc.kv_read_mxfp4(cache, pt, i32(lens), cum(new), rows=T)
    t = 0
    for b, n in enumerate(new):
        pos = torch.arange(before[b], lens[b], device="cuda")
        for part, x in enumerate((o["k"], o["v"])):
            w = ref.get(cache, pt, b, pos, part).float().bfloat16()
            assert torch.equal(x[t:t + n].nan_to_num(7.25), w.nan_to_num(7.25)) and torch.equal(x[t:t + n].isnan(), w.isnan())
        t += n


@pytest.mark.parametrize("B", [1, 31, 32, 33, 40, 1025, 2100])
def test_many_sequences(mhc, B):
    """A row finds its sequence whatever their number, empty ones among them."""
    g = torch.Generator().manual_seed(B)
    new = torch.randint(0, 3, (B,), generator=g).tolist()
    new[-1] = 2
    lens = [n + (b % 5) for b, n in enumerate(new)]
    pt, P = table(lens, 16)
    T = sum(new)
    x = torch.randn(2, T, 1, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(B)).bfloat16()
    cache = torch.full(mhc.kv_cache_shape(P, 1, 16, 64), 255, dtype=torch.uint8, device="cuda")
    mhc.kv_write_mxfp4(x[0], x[1], cache, pt, i32(lens), cum(new))
    o = mhc.kv_read_mxfp4(cache, pt, i32(lens), cum(new), rows=T)
    for i, n in enumerate(("k", "v")):
        want = ref.values4(*ref.quantize4(x[i].double(), 0))
        assert torch.equal(o[n].double(), want)


def test_places_that_do_not_exist(mhc):
    """Positions below 0, beyond the table, and pages outside the cache: nothing is written, NaN is read; rows outside
    every sequence are left as they were."""
    Hkv, D, page, P = 2, 128, 16, 5
    pt = i32([[0, 1], [2, -1], [7, 3], [4, 2147483647]])
    lens, new = [40, 30, 20, 3], [12, 8, 10, 5]              # b0: 28..39 (32.. beyond the table), b1: 22..29 on page -1 ...
    off = i32([2] + [2 + n for n in torch.tensor(new).cumsum(0).tolist()])
    T = 2 + sum(new) + 3
    x = torch.randn(2, T, Hkv, D, device="cuda", generator=torch.Generator("cuda").manual_seed(0))
    want = torch.full(mhc.kv_cache_shape(P, Hkv, page, D), 17, dtype=torch.uint8, device="cuda")
    cache = want.clone()
    mhc.kv_write_mxfp4(x[0], x[1], cache, pt, i32(lens), off)
    t, ok = 2, torch.zeros(T, dtype=torch.bool)
    for b, n in enumerate(new):
        for i in range(n):
            p = lens[b] - n + i
            if 0 <= p < 32 and 0 <= int(pt[b, p // 16]) < P:
                ok[t + i] = True
                for part in (0, 1):
                    ref.put(want, pt, b, torch.tensor([p], device="cuda"), part, *ref.quantize4(x[part, t + i:t + i + 1].double(), 0))
        t += n
    assert torch.equal(cache, want)
    o = {n: torch.full((T, Hkv, D), 3.0, device="cuda", dtype=torch.bfloat16) for n in ("k", "v")}
    mhc.kv_read_mxfp4(cache, pt, i32(lens), off, out=o)
    inside = torch.zeros(T, dtype=torch.bool)
    inside[2:2 + sum(new)] = True
    for part, n in enumerate(("k", "v")):
        assert bool((o[n][~inside] == 3.0).all())
        assert bool(o[n][inside & ~ok].isnan().all())
        assert torch.equal(o[n][ok].double(), ref.values4(*ref.quantize4(x[part][ok].double(), 0)))


def test_other_stream_and_replay(mhc):
    lens, new = [33, 70], [33, 7]
    pt, P = table(lens, 32)
    x = torch.randn(2, sum(new), 2, 64, device="cuda").bfloat16()
    cache = torch.zeros(mhc.kv_cache_shape(P, 2, 32, 64), dtype=torch.uint8, device="cuda")
    sl, off = i32(lens), cum(new)
    want = mhc.kv_write_mxfp4(x[0], x[1], cache.clone(), pt, sl, off)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    mhc.kv_write_mxfp4(x[0], x[1], cache, pt, sl, off, stream=s)
    o = mhc.kv_read_mxfp4(cache, pt, sl, off, rows=sum(new), stream=s)
    s.synchronize()
    assert torch.equal(cache, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mhc.kv_write_mxfp4(x[0], x[1], cache, pt, sl, off)
        again = mhc.kv_read_mxfp4(cache, pt, sl, off, rows=sum(new))
    x.neg_()
    off.copy_(cum([30, 8]))   # the graph reads the geometry when it runs
    graph.replay()
    torch.cuda.synchronize()
    w = mhc.kv_read_mxfp4(mhc.kv_write_mxfp4(x[0], x[1], want, pt, sl, off), pt, sl, off, rows=sum(new))
    assert torch.equal(cache, want) and torch.equal(again["k"][:38], w["k"][:38]) and torch.equal(again["v"][:38], w["v"][:38])
    assert not torch.equal(o["k"][:38], w["k"][:38])


def test_positions_past_32_bits_of_bytes(mhc):
    """A cache of more than 2^32 bytes: its last pages."""
    Hkv, D, page = 8, 128, 128
    P = (1 << 32) // (Hkv * 8 * 17 * D) + 40
    cache = torch.zeros(mhc.kv_cache_shape(P, Hkv, page, D), dtype=torch.uint8, device="cuda")
    assert cache.numel() > 1 << 32
    pt = i32([[P - 1, P - 3]])
    x = torch.randn(2, 200, Hkv, D, device="cuda").bfloat16()
    mhc.kv_write_mxfp4(x[0], x[1], cache, pt, i32([200]), i32([0, 200]))
    o = mhc.kv_read_mxfp4(cache, pt, i32([200]), i32([0, 200]), rows=200)
    assert torch.equal(o["v"].double(), ref.values4(*ref.quantize4(x[1].double(), 0)))
    assert torch.equal(ref.get(cache, pt, 0, torch.arange(200, device="cuda"), 0), ref.values4(*ref.quantize4(x[0].double(), 0)))
