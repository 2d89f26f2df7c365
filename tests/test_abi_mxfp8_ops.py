"""CPU-only checks of the MXFP8 operators' entry points: bad sizes, types, pointers, workspaces and overlaps are
refused before CUDA is touched, and empty calls launch nothing."""
import ctypes

import pytest

BASE = 0x100000000


def fake(i, off=0):
    return ctypes.c_void_p(BASE + i * (1 << 40) + off)


def norm(L, T=4, H=64, eps=1e-6, x=fake(0), res=fake(1), g=fake(2), ro=fake(3), li=fake(4), q=fake(5), s=fake(6), mode=0, block=32):
    return L.mhc_add_rmsnorm_mxfp8(x, res, g, T, H, eps, ro, li, q, s, mode, block, None)


def swiglu(L, T=4, F=64, gu=fake(0), q=fake(1), s=fake(2), mode=0, block=32):
    return L.mhc_swiglu_mxfp8(gu, T, F, q, s, mode, block, None)


def linear(L, T=4, K=64, N=16, x=fake(0), xs=fake(1), w=fake(2), sc=fake(3), st=0, out=fake(4), ot=0, ws=fake(5), wb=256):
    return L.mhc_linear_mxfp8(x, xs, w, sc, st, T, K, N, out, ot, ws, wb, None)


def experts(L, R=4, M=4, E=3, K=64, N=16, x=fake(0), xs=fake(1), rows=None, off=fake(6), w=fake(2), sc=fake(3), st=0, out=fake(4),
            ot=0, ws=fake(5), wb=256):
    return L.mhc_expert_linear_mxfp8(x, xs, R, rows, M, off, E, w, sc, st, K, N, out, ot, ws, wb, None)


@pytest.fixture(scope="module")
def L(mhc_lib):
    return mhc_lib.lib()


def refused(L, rc, text, status=-1):
    assert rc == status, rc
    assert text in L.mhc_last_error().decode(), L.mhc_last_error()


@pytest.mark.parametrize("kw,text", [
    ({"T": -1}, "T="), ({"T": (1 << 20) + 1}, "T="), ({"H": 12}, "H="), ({"H": 65544}, "H="), ({"H": 72}, "multiple of 32"),
    ({"eps": -1.0}, "rmsnorm_eps"), ({"eps": float("inf")}, "rmsnorm_eps"), ({"x": None}, "x is NULL"), ({"g": None}, "rmsnorm_weight"),
    ({"x": fake(0, 8)}, "aligned"), ({"res": fake(1, 2)}, "aligned"), ({"q": fake(5, 8)}, "aligned"), ({"q": None}, "layer_in_fp8"),
    ({"s": None}, "scales"), ({"mode": 2}, "scale mode"), ({"block": 64}, "scale_block"), ({"res": None}, "residual_out without"),
    ({"li": None, "q": None, "s": None}, "are NULL"), ({"li": fake(0)}, "overlaps an input"), ({"ro": fake(1, 16)}, "overlaps an input"),
    ({"q": fake(4, 64)}, "overlaps layer_in_fp8"), ({"s": fake(2)}, "overlaps an input")])
def test_norm_refusals(L, kw, text):
    refused(L, norm(L, **kw), text)


@pytest.mark.parametrize("kw,text", [
    ({"T": -1}, "T="), ({"F": 48}, "multiple of 32"), ({"F": 0}, "H="), ({"gu": None}, "gate_up"), ({"q": None}, "act_fp8"),
    ({"s": None}, "scales"), ({"mode": -1}, "scale mode"), ({"block": 0}, "scale_block"), ({"q": fake(0, 512)}, "overlaps an input")])
def test_swiglu_refusals(L, kw, text):
    refused(L, swiglu(L, **kw), text)


@pytest.mark.parametrize("kw,text", [
    ({"T": -1}, "rows"), ({"T": (1 << 20) + 1}, "rows"), ({"K": 16}, "K="), ({"K": 48}, "K="), ({"K": 65568}, "K="), ({"N": 4}, "N="),
    ({"N": 12}, "N="), ({"N": (1 << 20) + 8}, "N="), ({"st": 2}, "scale type"), ({"ot": 3}, "output type"), ({"x": None}, "x_fp8"),
    ({"xs": None}, "x_scales"), ({"w": None}, "w_fp8"), ({"sc": None}, "w_scales"), ({"out": None}, "out is NULL"),
    ({"x": fake(0, 4)}, "aligned"), ({"xs": fake(1, 1)}, "aligned"), ({"w": fake(2, 8)}, "aligned"), ({"out": fake(4, 2)}, "aligned"),
    ({"out": fake(0, 64)}, "overlaps an input"), ({"out": fake(3)}, "overlaps an input")])
@pytest.mark.parametrize("call", [linear, experts])
def test_product_refusals(L, call, kw, text):
    if call is experts and "T" in kw:
        kw = {"M": kw["T"], "R": kw["T"]}
    refused(L, call(L, **kw), text)


@pytest.mark.parametrize("kw,text", [
    ({"E": 0}, "E="), ({"E": 1025}, "E="), ({"off": None}, "expert_offsets"), ({"off": fake(6, 4)}, "aligned"), ({"R": 5}, "as many rows"),
    ({"rows": fake(7, 4)}, "aligned"), ({"R": 0, "rows": fake(7)}, "no rows"), ({"R": -1, "rows": fake(7)}, "rows"),
    ({"out": fake(7, 0), "rows": fake(7)}, "overlaps an input"), ({"out": fake(6)}, "overlaps an input")])
def test_expert_refusals(L, kw, text):
    refused(L, experts(L, **kw), text)


@pytest.mark.parametrize("call", [linear, experts])
def test_product_workspace_refusals(L, call):
    refused(L, call(L, ws=None), "workspace is NULL", -3)
    refused(L, call(L, ws=fake(5, 16)), "256-byte aligned", -3)
    refused(L, call(L, wb=255), "workspace has 255 bytes", -3)
    refused(L, call(L, ws=fake(0)), "workspace overlaps an input")
    refused(L, call(L, ws=fake(4)), "overlaps workspace")


def test_empty_calls_are_no_ops(L, mhc_lib):
    assert norm(L, T=0, x=None, g=None, q=None) == 0
    assert swiglu(L, T=0, gu=None) == 0
    assert linear(L, T=0, x=None, out=None, ws=None) == 0
    assert experts(L, R=0, M=0, x=None, out=None, ws=None) == 0
    assert mhc_lib.last_launch_count() == 0
    assert mhc_lib.linear_workspace_size() == 256


def test_binding_refuses_host_tensors(mhc_lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises((ValueError, RuntimeError)):
        mhc_lib.add_rmsnorm_mxfp8(x, x, x[0], rmsnorm_eps=1e-6)
    with pytest.raises((ValueError, RuntimeError)):
        mhc_lib.swiglu_mxfp8(x)
    q = torch.zeros((2, 64), dtype=torch.uint8)
    with pytest.raises((ValueError, RuntimeError)):
        mhc_lib.linear_mxfp8(q, torch.zeros(512, dtype=torch.uint8), q, torch.zeros((1, 1)), workspace=q)
    with pytest.raises((ValueError, RuntimeError)):
        mhc_lib.expert_linear_mxfp8(q, torch.zeros(512, dtype=torch.uint8), q[None], torch.zeros((1, 1, 1)), torch.zeros(2, dtype=torch.int32))


@pytest.mark.parametrize("off", [1, 2, 4, 8])
def test_misaligned_scale_outputs_are_refused(L, off):
    """The producers store four scale bytes as a word, so their scales are 16-byte aligned like every other pointer."""
    refused(L, norm(L, s=fake(6, off)), "layer_in_scales is not 16-byte aligned")
    refused(L, swiglu(L, s=fake(2, off)), "act_scales is not 16-byte aligned")
