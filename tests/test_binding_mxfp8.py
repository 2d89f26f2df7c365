"""CPU checks of the MXFP8 operators' binding: the calls run with their tensors' device current and on the right
stream, errors carry the library's status, and the argument checks name the argument."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import manifold_constrained_hyper_mhc_gb300 as mhc  # noqa: E402


class Stream:
    cuda_stream = 77


class FakeLib:
    """Stands in for the library: notes the current device of each call and returns `rc`."""

    def __init__(self, log, rc=0):
        self.log, self.rc = log, rc

    def mhc_linear_mxfp8(self, *args):
        self.log.append((torch.cuda.current_device(), args[-1]))
        return self.rc

    def mhc_last_error(self):
        return b"the reason"


@pytest.fixture
def fake(monkeypatch):
    state, log = {"device": 0}, []

    @contextlib.contextmanager
    def device(dev):
        before, state["device"] = state["device"], dev.index
        yield
        state["device"] = before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["device"])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(mhc, "_lib", FakeLib(log))
    return log


def test_a_call_runs_with_its_tensors_device_current(fake):
    mhc._run("mhc_linear_mxfp8", torch.device("cuda", 1), Stream(), 1, 2)
    mhc._run("mhc_linear_mxfp8", torch.device("cuda", 0), Stream(), 1, 2)
    assert fake == [(1, 77), (0, 77)] and torch.cuda.current_device() == 0


def test_without_a_stream_the_devices_current_one_is_used(fake, monkeypatch):
    if hasattr(torch._C, "_cuda_getCurrentRawStream"):
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index)
    else:
        monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: type("S", (), {"cuda_stream": 1000 + dev.index}))
    mhc._run("mhc_linear_mxfp8", torch.device("cuda", 1), None, 1)
    assert fake == [(1, 1001)]


def test_a_status_becomes_an_error_with_the_librarys_reason(fake, monkeypatch):
    monkeypatch.setattr(mhc._lib, "rc", -3)
    with pytest.raises(mhc.MhcError, match="mhc_linear_mxfp8: MHC_ERR_WORKSPACE .the reason."):
        mhc._run("mhc_linear_mxfp8", torch.device("cuda", 0), Stream())


def test_argument_checks_name_the_argument():
    bf16, fp8, e8m0, f32, i32 = mhc._dtypes()
    cpu = torch.device("cpu")
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    assert mhc._arg(x, "x", bf16, (2, 64), cpu) == x.data_ptr()
    with pytest.raises(TypeError, match="x must be bfloat16 or int16 or uint16, got torch.float32"):
        mhc._arg(x.float(), "x", bf16, (2, 64), cpu)
    with pytest.raises(ValueError, match=r"x has shape \(2, 64\), expected \(2, 32\)"):
        mhc._arg(x, "x", bf16, (2, 32), cpu)
    with pytest.raises(ValueError, match="x must be a contiguous tensor on cpu"):
        mhc._arg(torch.zeros((64, 2), dtype=torch.bfloat16).t(), "x", bf16, (2, 64), cpu)
    with pytest.raises(ValueError, match="x must be a contiguous tensor on cuda:1"):
        mhc._arg(x, "x", bf16, (2, 64), torch.device("cuda", 1))
    with pytest.raises(ValueError, match="gate_up must be a contiguous CUDA tensor"):
        mhc._cuda(x, "gate_up")


@pytest.mark.parametrize("rows,cols", [(0, 32), (1, 32), (128, 128), (129, 160), (6, 7168), (300, 4064)])
def test_scale_shape_is_the_librarys(mhc_lib, rows, cols):
    assert mhc._scale_shape(rows, cols) == (mhc.mxfp8_scale_bytes(rows, cols),)
    assert mhc._scale_shape(rows, cols + 8) == (0,)


@pytest.mark.parametrize("zero", [False, True])
def test_new_tensors_belong_to_the_calls_stream(monkeypatch, zero):
    on = []

    @contextlib.contextmanager
    def use(stream):
        on.append(stream)
        yield

    monkeypatch.setattr(torch.cuda, "stream", use)
    s = Stream()
    t = mhc._new((2, 3), torch.uint8, torch.device("cpu"), s, zero=zero)
    assert on == [s] and t.shape == (2, 3) and t.dtype == torch.uint8
    mhc._new((2, 3), torch.uint8, torch.device("cpu"), None)
    assert on == [s]
