"""GPU checks of which rows of the prompt attention a value of v that is not finite sends the plain way: those beside a row
that sees it and does not see it, and no others (the others keep their bits)."""
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


def make(mhc, n, L, D, G, Hkv, dev="cuda"):
    g = torch.Generator(device=dev).manual_seed(D + L)
    q, k, v = (torch.randn(t, h, D, generator=g, device=dev).bfloat16() for t, h in ((n, G * Hkv), (L, Hkv), (L, Hkv)))
    offsets = [torch.tensor([0, t], dtype=torch.int32, device=dev) for t in (n, L)]
    ws = torch.zeros(mhc.prompt_workspace_size(), dtype=torch.uint8, device=dev)
    return q, k, v, lambda v: mhc.prompt_attention(q, k, v, *offsets, workspace=ws)["attn_out"]


def held(q, k, v, rows, L, o, scale):
    """Those rows within the bound, each over the keys that it sees."""
    n = q.shape[0]
    for r in rows:
        end = L - n + r + 1
        out, _, tol, _ = ref.attend(q[r:r + 1], k[:end].double(), v[:end].double(), scale, "bf16")
        ref.check_out(o[r:r + 1], out, tol)


@pytest.mark.parametrize("D,G,Hkv", [(128, 4, 2), (64, 4, 1), (64, 1, 2), (128, 7, 1)])
@pytest.mark.parametrize("prefix", [0, 333])
def test_later_tokens_leave_the_pairs_before_their_bits(mhc, D, G, Hkv, prefix):
    """The first pair of row tiles ends before the token: none of its rows sees it, and nothing of them changes."""
    pair = 2 * (128 // G)
    n = pair + 40
    q, k, v, call = make(mhc, n, prefix + n, D, G, Hkv)
    clean = call(v)
    bad = v.clone()
    bad[prefix + pair, 0, 3] = math.inf         # the first token behind it
    o = call(bad)
    assert torch.equal(o[:pair], clean[:pair])
    assert bool((~o[pair:, :G, 3].isfinite()).all()) and bool(o[pair:, :G, 4:].isfinite().all())
    bad = v.clone()
    bad[prefix + pair + 20, 0, 3] = math.nan
    o = call(bad)
    assert torch.equal(o[:pair], clean[:pair])
    held(q, k, v, range(pair, pair + 20), prefix + n, o, D ** -0.5)


@pytest.mark.parametrize("D,G,Hkv", [(128, 4, 2), (64, 8, 1), (128, 1, 1)])
def test_a_value_that_all_rows_see_is_no_reason(mhc, D, G, Hkv):
    """The last key of the prefix, in a tile of keys that is seen in part: its column is not finite, the others keep their bits."""
    n, prefix = 2 * (128 // G), 200
    q, k, v, call = make(mhc, n, prefix + n, D, G, Hkv)
    clean = call(v)
    bad = v.clone()
    bad[prefix, 0, 3] = math.inf                # (the first new token sees it, itself)
    o = call(bad)
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[:, :G, 3] = True
    assert bool((~o[hit].isfinite()).all()) and torch.equal(o[~hit], clean[~hit])


@pytest.mark.parametrize("D,G,Hkv", [(128, 4, 2), (64, 8, 1), (128, 1, 1)])
@pytest.mark.parametrize("prefix", [0, 100])
def test_both_tiles_of_a_pair(mhc, D, G, Hkv, prefix):
    """A token of the first and one of the second tile: every row that does not see it is within its bound."""
    tile = 128 // G
    n = 2 * tile
    q, k, v, call = make(mhc, n, prefix + n, D, G, Hkv)
    for at in (tile // 2, tile - 1, tile, tile + tile // 2, n - 1):
        bad = v.clone()
        bad[prefix + at, 0, 3] = -math.inf
        o = call(bad)
        held(q, k, v, range(0, at, max(1, at // 20)), prefix + n, o, D ** -0.5)
        assert bool((~o[at:, :G, 3].isfinite()).all()) and bool(o[at:, :G, 4:].isfinite().all())
