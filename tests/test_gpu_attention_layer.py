"""The attention operators as a decoder uses them: the fused step's MXFP8 layer input through the q/k/v product, the cache
write, the attention (of whole prompts, of a later chunk after its prefix read back from the cache, and of new tokens over
the cache) with an MXFP8 result, and the output product, whose result is the next fused step's layer output.

Each operator is held to its 64-bit definition on the inputs it got (the single operators' bounds); a whole step runs
captured in one graph and gives the same bits as call by call."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import _attention as ref  # noqa: E402
import _mxfp8 as mx  # noqa: E402
from manifold_constrained_hyper_mhc_gb300 import synth  # noqa: E402
from test_gpu_linear_mxfp8 import check as check_linear  # noqa: E402

pytestmark = pytest.mark.gpu
SC = synth.scalars()
H, PAGE = 1024, 32


@pytest.fixture(scope="module")
def mhc(mhc_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return mhc_lib


def dev(a):
    if a.dtype == np.uint16:
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda().view(torch.bfloat16)
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cum(v):
    return i32([0] + torch.tensor(v).cumsum(0).tolist())


class Layer:
    def __init__(self, mhc, Hq, Hkv, D, wide):
        self.mhc, self.Hq, self.Hkv, self.D, self.wide = mhc, Hq, Hkv, D, wide
        w = synth.Workload("attention layer", 8, H, 5)
        self.phi, self.bias, self.ms, self.gamma = map(dev, synth.weights(w))
        self.wq, self.ws = mx.weights((), (Hq + 2 * Hkv) * D, H, 1, wide)
        self.ws = self.ws * 2.0 ** -3 if wide else self.ws - 3   # scores of a few units
        self.oq, self.os = mx.weights((), H, Hq * D, 2, wide)
        self.decode_ws = torch.zeros(mhc.decode_workspace_size(), dtype=torch.uint8, device="cuda")

    def tokens(self, T, seed):
        w = synth.Workload("attention layer", T, H, seed)
        return tuple(map(dev, synth.tokens(w)))

    def qkv(self, a, ws):
        x = self.mhc.linear_mxfp8(a["layer_in_fp8"], a["layer_in_scales"], self.wq, self.ws, workspace=ws).view(-1, self.Hq + 2 * self.Hkv, self.D)
        return x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]

    def step(self, R, Y, pp, pc, ws, attend):
        """The fused step, attend(q, k, v) and the output product, then the next fused step."""
        mhc = self.mhc
        a = mhc.shifted_post_pre_mxfp8(R, Y, pp, pc, self.phi, self.bias, self.ms, self.gamma, **SC, want_bf16=False, workspace=ws)
        q, k, v = self.qkv(a, ws)
        o = attend(q, k, v)
        y = mhc.linear_mxfp8(o["attn_fp8"], o["attn_scales"], self.oq, self.os, workspace=ws)
        b = mhc.shifted_post_pre(a["residual_out"], y, a["post_mix"], a["comb_res_mix"], self.phi, self.bias, self.ms, self.gamma, **SC, workspace=ws)
        return a, (q, k, v), o, y, b


@pytest.mark.parametrize("Hq,Hkv,D,wide", [(8, 2, 128, False), (12, 4, 64, True)])
def test_a_prompt_a_later_chunk_and_new_tokens(mhc, Hq, Hkv, D, wide):
    m = Layer(mhc, Hq, Hkv, D, wide)
    first, second, new = [70, 1, 200], [40, 130, 3], [1, 6, 2]
    total = [a + b + c for a, b, c in zip(first, second, new)]
    W = max(-(-n // PAGE) for n in total)
    P = 3 * W + 1
    order = torch.randperm(P, generator=torch.Generator().manual_seed(3)).int().cuda()
    table = order[:3 * W].view(3, W).contiguous()
    cache = torch.full(mhc.kv_cache_shape(P, Hkv, PAGE, D), 255, dtype=torch.uint8, device="cuda")

    def values(part, b, n):
        return ref.get(cache, table, b, torch.arange(n, device="cuda"), part)

    # ---- the prompts
    n1, lens1 = sum(first), i32(first)
    ws = mhc.new_workspace(max(n1, sum(second)), H)

    def prompt(q, k, v):
        mhc.kv_write_mxfp4(k, v, cache, table, lens1, cum(first))
        return mhc.prompt_attention(q, k, v, cum(first), cum(first), want_mxfp8=True, workspace=ws)
    a, (q, k, v), o, y, b = m.step(*m.tokens(n1, 1), ws, prompt)
    mhc.check_status(ws)
    parts, t = [], 0
    for i, n in enumerate(first):
        for part, x in enumerate((k, v)):
            assert torch.equal(values(part, i, n), ref.values4(*ref.quantize4(x[t:t + n].double(), 0)))
        parts.append(ref.attend(q[t:t + n], k[t:t + n].double(), v[t:t + n].double(), D ** -0.5, "bf16"))
        ref.check_out(o["attn_out"][t:t + n], parts[-1][0], parts[-1][2])
        t += n
    ref.check_mx(o["attn_fp8"], o["attn_scales"], torch.cat([p[0] for p in parts]).flatten(1), torch.cat([p[2] for p in parts]).flatten(1))
    check_linear(y, mx.dequant_x(o["attn_fp8"], o["attn_scales"]), mx.dequant_w(m.oq, m.os))
    assert bool(b["layer_in"].isfinite().all())

    # ---- the next chunks: their prefixes read back in front of their own keys
    both = [x + z for x, z in zip(first, second)]
    n2, lens2 = sum(second), i32(both)

    def chunk(q, k, v):
        old = mhc.kv_read_mxfp4(cache, table, lens1, cum(first), rows=n1)
        mhc.kv_write_mxfp4(k, v, cache, table, lens2, cum(second))
        kk, vv = [torch.cat([z for i in range(3) for z in (p[sum(first[:i]):sum(first[:i + 1])], x[sum(second[:i]):sum(second[:i + 1])])])
                  for p, x in ((old["k"], k), (old["v"], v))]
        return {**mhc.prompt_attention(q, kk, vv, cum(second), cum(both), want_mxfp8=True, workspace=ws), "k": kk, "v": vv}
    a, (q, k, v), o, y, b = m.step(*m.tokens(n2, 2), ws, chunk)
    t = j = 0
    for i, n in enumerate(second):
        L = both[i]
        assert torch.equal(o["k"][j:j + first[i]].double(), values(0, i, first[i]))
        want, _, tol, _ = ref.attend(q[t:t + n], o["k"][j:j + L].double(), o["v"][j:j + L].double(), D ** -0.5, "bf16")
        ref.check_out(o["attn_out"][t:t + n], want, tol)
        t, j = t + n, j + L

    # ---- new tokens, captured: one of the first sequence, a verify block of the second, two of the third
    n3, lens3 = sum(new), i32(total)
    inputs = m.tokens(n3, 3)
    off = cum(new)

    def decode(q, k, v):
        mhc.kv_write_mxfp4(k, v, cache, table, lens3, off, scale_mode=mhc.MX_SCALE_CEIL)
        return mhc.decode_attention_mxfp4(q, cache, table, lens3, off, want_mxfp8=True, want_lse=True, workspace=m.decode_ws)
    a, (q, k, v), o, y, b = m.step(*inputs, ws, decode)
    mhc.check_status(m.decode_ws)
    parts, t = [], 0
    for i, n in enumerate(new):
        assert torch.equal(values(0, i, total[i])[both[i]:], ref.values4(*ref.quantize4(k[t:t + n].double(), 1)))
        parts.append(ref.attend(q[t:t + n], values(0, i, total[i]), values(1, i, total[i]), D ** -0.5, "f16"))
        ref.check_out(o["attn_out"][t:t + n], parts[-1][0], parts[-1][2])
        ref.check_lse(o["lse"][t:t + n], parts[-1][1], parts[-1][3])
        t += n
    ref.check_mx(o["attn_fp8"], o["attn_scales"], torch.cat([p[0] for p in parts]).flatten(1), torch.cat([p[2] for p in parts]).flatten(1))
    check_linear(y, mx.dequant_x(o["attn_fp8"], o["attn_scales"]), mx.dequant_w(m.oq, m.os))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = m.step(*inputs, ws, decode)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again[3].view(torch.int16), y.view(torch.int16)) and torch.equal(again[4]["layer_in"].view(torch.int16), b["layer_in"].view(torch.int16))


def test_two_parts_joined_by_their_log_sums(mhc):
    """The log-sums' use: a prompt's attention to a shared prefix and to its own keys, each alone, joined."""
    D, Hq, Hkv, n, L = 64, 4, 2, 50, 300
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, D, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k, v = r(n, Hq), r(L + n, Hkv), r(L + n, Hkv)
    whole = mhc.prompt_attention(q, k, v, cum([n]), cum([L + n]), want_lse=True)
    own = mhc.prompt_attention(q, k[L:], v[L:], cum([n]), cum([n]), want_lse=True)
    # (every row sees the whole prefix: each row as a sequence of its own)
    rows = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    kp, vp = k[:L].repeat(n, 1, 1), v[:L].repeat(n, 1, 1)
    pre = mhc.prompt_attention(q, kp, vp, rows, rows * L, want_lse=True)
    m = torch.maximum(own["lse"], pre["lse"])
    a, b = torch.exp(own["lse"] - m), torch.exp(pre["lse"] - m)
    out = (own["attn_out"].double() * a[..., None] + pre["attn_out"].double() * b[..., None]) / (a + b)[..., None]
    want, lse, tol, tol_lse = ref.attend(q, k.double(), v.double(), D ** -0.5, "bf16")
    scale = torch.maximum(own["attn_out"].double().abs(), pre["attn_out"].double().abs())
    assert bool(((out - want).abs() <= 4 * tol + 2.0 ** -8 * scale).all())   # (each part rounded once more, to bf16)
    assert bool(((m + torch.log(a + b) - lse).abs() <= 4 * tol_lse + 2.0 ** -20).all())
    ref.check_lse(whole["lse"], lse, tol_lse)
