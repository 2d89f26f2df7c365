"""CPU-only checks of the attention operators' entry points: bad sizes, strides, types, pointers, workspaces and overlaps
are refused before CUDA is touched, and empty calls launch nothing."""
import ctypes

import pytest

BASE = 0x100000000


def fake(i, off=0):
    return ctypes.c_void_p(BASE + i * (1 << 44) + off)


def write(L, T=4, B=2, W=3, pages=5, Hkv=2, page=16, D=64, k=fake(0), v=fake(1), ks=128, vs=128, ty=0, off=fake(2), sl=fake(3), pt=fake(4), cache=fake(5), mode=0):
    return L.mhc_kv_write_mxfp4(k, v, ty, ks, vs, T, off, sl, pt, B, W, cache, pages, Hkv, page, D, mode, None)


def read(L, T=4, B=2, W=3, pages=5, Hkv=2, page=16, D=64, k=fake(0), v=fake(1), off=fake(2), sl=fake(3), pt=fake(4), cache=fake(5)):
    return L.mhc_kv_read_mxfp4(cache, pages, Hkv, page, D, off, sl, pt, B, W, T, k, v, None)


def decode(L, T=4, B=2, W=3, pages=5, Hq=4, Hkv=2, page=16, D=64, q=fake(0), qs=256, off=fake(2), sl=fake(3), pt=fake(4), cache=fake(5), scale=0.1,
           out=fake(6), fp8=fake(7), tiles=fake(8), mode=0, lse=fake(9), ws=fake(10), wb=1 << 30):
    return L.mhc_decode_attention_mxfp4(q, qs, T, Hq, off, sl, pt, B, W, cache, pages, Hkv, page, D, scale, out, fp8, tiles, mode, lse, ws, wb, None)


def prompt(L, T=4, Tk=4, B=2, Hq=4, Hkv=2, D=64, q=fake(0), qs=256, k=fake(1), ks=128, v=fake(5), vs=128, off=fake(2), koff=fake(3), scale=0.1,
           out=fake(6), fp8=fake(7), tiles=fake(8), mode=0, lse=fake(9), ws=fake(10), wb=256):
    return L.mhc_prompt_attention(q, qs, k, ks, v, vs, T, Tk, Hq, Hkv, D, off, koff, B, scale, out, fp8, tiles, mode, lse, ws, wb, None)


@pytest.fixture(scope="module")
def L(mhc_lib):
    return mhc_lib.lib()


def refused(L, rc, text, status=-1):
    assert rc == status, rc
    assert text in L.mhc_last_error().decode(), L.mhc_last_error()


CACHE = [({"T": -1}, "T="), ({"T": (1 << 20) + 1}, "T="), ({"B": -1}, "B="), ({"B": (1 << 16) + 1}, "B="), ({"W": 0}, "table_width"),
         ({"W": (1 << 26) + 1}, "table_width"), ({"pages": 0}, "pages="), ({"pages": 1 << 31}, "pages="), ({"page": 8}, "page_size"),
         ({"page": 48}, "page_size"), ({"page": 512}, "page_size"), ({"D": 32}, "head_dim"), ({"D": 96}, "head_dim"), ({"D": 256}, "head_dim"),
         ({"Hkv": 0}, "kv_heads"), ({"Hkv": 1025}, "kv_heads"), ({"off": None}, "offsets is NULL"), ({"sl": None}, "seq_lens is NULL"),
         ({"pt": None}, "page_table is NULL"), ({"off": fake(2, 2)}, "offsets is not 4-byte"), ({"cache": None}, "cache is NULL"),
         ({"cache": fake(5, 8)}, "cache is not 16-byte")]


@pytest.mark.parametrize("call", [write, read, decode])
@pytest.mark.parametrize("kw,text", CACHE)
def test_cache_refusals(L, call, kw, text):
    refused(L, call(L, **kw), text)


@pytest.mark.parametrize("kw,text", [
    ({"k": None}, "k is NULL"), ({"v": fake(1, 8)}, "v is not 16-byte"), ({"ty": 2}, "value type"), ({"mode": 2}, "scale mode"), ({"ks": 120}, "k_stride"),
    ({"vs": 132}, "v_stride"), ({"ks": 1 << 31}, "k_stride"), ({"cache": fake(0, 64)}, "cache overlaps"), ({"cache": fake(4)}, "cache overlaps")])
def test_write_refusals(L, kw, text):
    refused(L, write(L, **kw), text)


@pytest.mark.parametrize("kw,text", [({"k": None}, "k_out is NULL"), ({"v": fake(1, 4)}, "v_out is not 16-byte"), ({"k": fake(1, 256)}, "k_out overlaps v_out"),
                                     ({"v": fake(5, 160)}, "v_out overlaps an input"), ({"k": fake(3)}, "k_out overlaps an input")])
def test_read_refusals(L, kw, text):
    refused(L, read(L, **kw), text)


@pytest.mark.parametrize("call", [decode, prompt])
@pytest.mark.parametrize("kw,text", [
    ({"Hq": 3}, "q_heads"), ({"Hq": 0}, "q_heads"), ({"Hq": 130}, "q_heads"), ({"Hq": 2048, "qs": 1 << 17}, "q_heads"), ({"D": 72}, "head_dim"),
    ({"qs": 248}, "q_stride"), ({"qs": 260}, "q_stride"), ({"scale": float("nan")}, "sm_scale"), ({"scale": float("inf")}, "sm_scale"),
    ({"q": None}, "q is NULL"), ({"q": fake(0, 2)}, "q is not 16-byte"), ({"out": None, "fp8": None, "tiles": None}, "are NULL"),
    ({"tiles": None}, "attn_scales is NULL"), ({"fp8": None}, "attn_fp8 is NULL"), ({"mode": 7}, "scale mode"), ({"out": fake(6, 8)}, "attn_out is not"),
    ({"lse": fake(9, 2)}, "lse is not"), ({"out": fake(0, 256)}, "attn_out overlaps an input"), ({"lse": fake(6)}, "attn_out overlaps lse"),
    ({"fp8": fake(2)}, "attn_fp8 overlaps an input"), ({"ws": fake(7)}, "overlaps workspace")])
def test_attention_refusals(L, call, kw, text):
    refused(L, call(L, **kw), text)


@pytest.mark.parametrize("call", [decode, prompt])
@pytest.mark.parametrize("kw,text", [({"ws": None}, "workspace is NULL"), ({"ws": fake(10, 128)}, "256-byte"), ({"wb": 255}, "needs")])
def test_workspaces(L, call, kw, text):
    refused(L, call(L, **kw), text, -3)


@pytest.mark.parametrize("kw,text", [
    ({"Tk": -1}, "Tk="), ({"Tk": (1 << 20) + 1}, "Tk="), ({"T": -1}, "Tq="), ({"B": -1}, "B="), ({"k": None}, "k is NULL"), ({"v": None}, "v is NULL"),
    ({"ks": 64}, "k_stride"), ({"vs": 129}, "v_stride"), ({"koff": None}, "k_offsets"), ({"off": fake(2, 1)}, "q_offsets"), ({"out": fake(5)}, "overlaps an input")])
def test_prompt_refusals(L, kw, text):
    refused(L, prompt(L, **kw), text)


@pytest.mark.parametrize("call", [write, read, decode, prompt])
@pytest.mark.parametrize("kw", [{"T": 0}, {"B": 0}, {"T": 0, "B": 0}])
def test_empty_calls(L, call, kw):
    assert call(L, **kw) == 0 and L.mhc_last_launch_count() == 0


def test_cache_bytes(L, mhc_lib):
    for P, H, page, D in [(1, 1, 16, 64), (7, 3, 64, 128), (1000, 8, 256, 128)]:
        shape = mhc_lib.kv_cache_shape(P, H, page, D)
        assert L.mhc_kv_cache_bytes(P, H, page, D) == shape[0] * shape[1] * shape[2] * shape[3] == P * H * page * 17 * D // 16
    assert L.mhc_kv_cache_bytes(1, 1, 17, 64) == 0 and L.mhc_kv_cache_bytes(0, 1, 16, 64) == 0
    for bad in [(1, 1, 17, 64), (1, 1, 16, 80), (0, 1, 16, 64), (1, 0, 16, 64)]:
        with pytest.raises(ValueError):
            mhc_lib.kv_cache_shape(*bad)
