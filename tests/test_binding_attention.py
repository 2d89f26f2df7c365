"""CPU checks of the attention operators' binding: which tensors are taken, and that a refusal names the argument."""
import pytest

torch = pytest.importorskip("torch")

import manifold_constrained_hyper_mhc_gb300 as mhc  # noqa: E402

CPU = torch.device("cpu")
BF16 = (torch.bfloat16,)


def test_rows_may_be_parts_of_wider_rows():
    wide = torch.zeros(5, 8, 64, dtype=torch.bfloat16)
    q = wide[:, 2:5]
    assert mhc._rows(q, "q", BF16, (5, 3, 64), CPU) == (wide.data_ptr() + 2 * 64 * 2, 8 * 64)
    assert mhc._rows(wide[:, 3:4], "q", BF16, (5, 1, 64), CPU)[1] == 8 * 64
    assert mhc._rows(wide[:1], "q", BF16, (1, 8, 64), CPU)[1] == 8 * 64          # one row: any distance
    assert mhc._rows(wide[4:5, :2], "q", BF16, (1, 2, 64), CPU)[1] == 2 * 64
    assert mhc._rows(torch.zeros(64, 3, 4, dtype=torch.bfloat16)[:0].permute(0, 1, 2), "q", BF16, (0, 3, 4), CPU)[1] == 12


@pytest.mark.parametrize("t,what", [
    (torch.zeros(5, 3, 64), "q must be bfloat16, got torch.float32"),
    (torch.zeros(5, 2, 64, dtype=torch.bfloat16), r"q has shape \(5, 2, 64\), expected \(5, 3, 64\)"),
    (torch.zeros(5, 64, 3, dtype=torch.bfloat16).transpose(1, 2), "heads lie next to each other"),
    (torch.zeros(5, 6, 64, dtype=torch.bfloat16)[:, ::2], "heads lie next to each other"),
    (torch.zeros(3, 5, 64, dtype=torch.bfloat16).transpose(0, 1), "heads lie next to each other"),
    (torch.zeros(5, 3, 128, dtype=torch.bfloat16)[..., ::2], "heads lie next to each other")])
def test_other_rows_are_refused(t, what):
    with pytest.raises((TypeError, ValueError), match=what):
        mhc._rows(t, "q", BF16, (5, 3, 64), CPU)


def test_sizes_are_three():
    assert tuple(mhc._three(torch.zeros(2, 3, 4), "k")) == (2, 3, 4)
    with pytest.raises(ValueError, match=r"k has shape \(2, 12\), expected \[tokens, heads, head_dim\]"):
        mhc._three(torch.zeros(2, 12), "k")


def test_a_cache_on_the_cpu_is_refused():
    with pytest.raises(ValueError, match="cache must be a contiguous CUDA tensor"):
        mhc.kv_read_mxfp4(torch.zeros(1, 1, 1, 1088, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                          torch.zeros(2, dtype=torch.int32), rows=1)


def test_workspace_sizes(mhc_lib):
    assert mhc_lib.prompt_workspace_size() == mhc_lib.linear_workspace_size() and mhc_lib.decode_workspace_size() > 1 << 20
