"""The 8-bit operators as a decoder uses them together: the fused step's MXFP8 layer input through the experts
(gate/up product with the rows taken by index, SwiGLU, down product, the experts' sum as the next layer output) into the
next fused step, then the final norm and the head's product.

Each operator is held to its 64-bit definition on the actual inputs it got, so the tolerances are the single operators'
(stated in their tests); the whole chain runs captured in one graph and gives the same bits as call by call."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import _mxfp8 as ref  # noqa: E402
from manifold_constrained_hyper_mhc_gb300 import synth  # noqa: E402
from test_gpu_linear_mxfp8 import check  # noqa: E402
from test_gpu_norm_mxfp8 import check_mx, norm_ref  # noqa: E402

pytestmark = pytest.mark.gpu
SC = synth.scalars()


@pytest.fixture(scope="module")
def mhc(mhc_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return mhc_lib


def dev(a):
    if a.dtype == np.uint16:
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda().view(torch.bfloat16)
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("T,wide", [(1, False), (6, True), (150, False), (400, True)])
def test_a_layer_of_experts_between_two_fused_steps(mhc, T, wide):
    H, F, E, topk, V = 1024, 288, 8, 3, 1000
    w = synth.Workload("layer", T, H, 40 + T)
    phi, bias, ms, gamma = map(dev, synth.weights(w))
    R, Y, pp, pc = map(dev, synth.tokens(w))
    gq, gs = ref.weights((E,), 2 * F, H, 1, wide)
    dq, ds = ref.weights((E,), H, F, 2, wide)
    hq, hs = ref.weights((), V, H, 3, wide)
    gen = torch.Generator(device="cuda").manual_seed(T)
    pick = torch.rand(T, E, generator=gen, device="cuda").topk(topk, 1)
    order = torch.argsort(pick.indices.reshape(-1), stable=True)
    rows = (order // topk).int()
    off = torch.cat([torch.zeros(1, device="cuda"), torch.bincount(pick.indices.reshape(-1), minlength=E).cumsum(0)]).int()
    prob = torch.softmax(pick.values, 1)
    back = torch.argsort(order).view(T, topk)
    ws = mhc.new_workspace(T, H)

    def layer():
        a = mhc.shifted_post_pre_mxfp8(R, Y, pp, pc, phi, bias, ms, gamma, **SC, want_bf16=False, workspace=ws)
        up = mhc.expert_linear_mxfp8(a["layer_in_fp8"], a["layer_in_scales"], gq, gs, off, rows=rows, workspace=ws)
        act = mhc.swiglu_mxfp8(up, scale_mode=mhc.MX_SCALE_CEIL, scale_block=128)
        down = mhc.expert_linear_mxfp8(act["act_fp8"], act["act_scales"], dq, ds, off, workspace=ws)
        y = (down[back].float() * prob[:, :, None]).sum(1).bfloat16()
        b = mhc.shifted_post_pre(a["residual_out"], y, a["post_mix"], a["comb_res_mix"], phi, bias, ms, gamma, **SC, workspace=ws)
        n = mhc.add_rmsnorm_mxfp8(b["layer_in"], y, gamma, rmsnorm_eps=SC["rmsnorm_eps"], want_bf16=True)
        logits = mhc.linear_mxfp8(n["layer_in_fp8"], n["layer_in_scales"], hq, hs, out_dtype=torch.float32, workspace=ws)
        return a, up, act, down, y, b, n, logits

    a, up, act, down, y, b, n, logits = layer()
    mhc.check_status(ws)
    x = ref.dequant_x(a["layer_in_fp8"], a["layer_in_scales"])
    o = off.tolist()
    xa = ref.dequant_x(act["act_fp8"], act["act_scales"])
    for e in range(E):
        r = slice(o[e], o[e + 1])
        if o[e + 1] > o[e]:
            check(up[r], x[rows[r].long()], ref.dequant_w(gq[e], gs[e]))
            check(down[r], xa[r], ref.dequant_w(dq[e], ds[e]))
    g, u = up[:, :F].double(), up[:, F:].double()
    check_mx(act["act_fp8"], act["act_scales"], g / (1 + torch.exp(-g)) * u, 128, 1, exact_subnormals=False)
    assert bool(b["layer_in"].isfinite().all())
    want = norm_ref(n["residual_out"], gamma, SC["rmsnorm_eps"])
    assert bool(((n["layer_in"].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -19) * want.abs() + 2.0 ** -133).all())
    check(logits, ref.dequant_x(n["layer_in_fp8"], n["layer_in_scales"]), ref.dequant_w(hq, hs))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = layer()
    graph.replay()
    torch.cuda.synchronize()
    mhc.check_status(ws)
    assert torch.equal(again[-1], logits) and torch.equal(again[4].view(torch.int16), y.view(torch.int16))
