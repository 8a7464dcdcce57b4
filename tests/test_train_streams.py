"""How the training operators hand memory over to another stream, without a
GPU: stand-in streams and tensors say which object waits and what is recorded."""
import pytest
import torch

import swiglu_activation_cast_amd._train_binding as tb

DEV = torch.device("cuda", 0)


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle
        self.waited = []

    def wait_stream(self, other):
        self.waited.append(other)


class Tensor:
    def __init__(self):
        self.recorded = []

    def record_stream(self, stream):
        self.recorded.append(stream)


@pytest.fixture
def streams(monkeypatch):
    """The default stream, another one that is current, and a third."""
    s = {"default": Stream(0), "current": Stream(0x1000), "third": Stream(0x2000)}
    made = {}

    def external(handle, device=None):
        # torch takes a null handle as none given and makes a new stream
        return made.setdefault(handle, Stream(handle if handle else 0x9999))

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: s["current"])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: s["default"])
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    s["made"] = made
    return s


@pytest.mark.parametrize("as_handle", [False, True])
def test_the_default_stream_itself_waits_and_is_recorded(streams, as_handle):
    t = Tensor()
    tb._other_stream(DEV, 0 if as_handle else streams["default"], t, None)
    assert streams["default"].waited == [streams["current"]] and t.recorded == [streams["default"]]
    assert not streams["made"]


@pytest.mark.parametrize("as_handle", [False, True])
def test_any_other_stream_waits_and_is_recorded(streams, as_handle):
    t = Tensor()
    tb._other_stream(DEV, 0x2000 if as_handle else streams["third"], None, t)
    other = streams["made"][0x2000] if as_handle else streams["third"]
    assert other.waited == [streams["current"]] and t.recorded == [other]
    assert len(streams["made"]) == as_handle


@pytest.mark.parametrize("as_handle", [False, True])
def test_the_current_stream_needs_nothing(streams, as_handle):
    t = Tensor()
    tb._other_stream(DEV, 0x1000 if as_handle else streams["current"], t)
    assert not streams["current"].waited and not t.recorded and not streams["made"]


# every call of the binding with a stream, on CPU stand-ins: inputs, outputs and
# workspace
def _ln():
    return torch.randn(8, 16), torch.randn(16), torch.randn(16), torch.randn(8), torch.rand(8)


def call_ln_fwd():
    x, w, b, mean, rstd = _ln()
    return [x, w, b], tb.mxtrain_layer_norm_fwd(x, w, b, stream=7)


def call_ln_bwd():
    x, w, _, mean, rstd = _ln()
    dy, ws = torch.randn(8, 16), torch.empty(64, dtype=torch.uint8)
    return [dy, x, mean, rstd, w, ws], tb.mxtrain_layer_norm_bwd(dy, x, mean, rstd, w, workspace=ws, stream=7)


def _experts():
    a, dy = torch.zeros((16, 24), dtype=torch.bfloat16), torch.zeros((16, 32), dtype=torch.bfloat16)
    return a, dy, torch.zeros((2, 32, 24), dtype=torch.bfloat16), torch.tensor([3, 16], dtype=torch.int32)


def call_gemm():
    a, _, b, ends = _experts()
    return [a, b, ends], (tb.mxtrain_grouped_gemm(a, b, ends, stream=7),)


def call_gemm_k():
    a, dy, _, ends = _experts()
    return [dy, a, ends], (tb.mxtrain_grouped_gemm_k(dy, a, ends, stream=7),)


def call_newton_schulz():
    g = torch.randn(2, 8, 16)
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    return [g, ws], (tb.mxtrain_newton_schulz(g, workspace=ws, stream=7),)


@pytest.mark.parametrize("call", [call_ln_fwd, call_ln_bwd, call_gemm, call_gemm_k, call_newton_schulz])
def test_everything_a_call_touches_is_recorded_on_its_stream(monkeypatch, call):
    """An input that the caller drops right after the call goes back to the
    current stream's pool, like an output or the workspace."""
    recorded = []
    monkeypatch.setattr(tb, "_gpu", lambda t, *a, **k: t)
    monkeypatch.setattr(tb, "_call", lambda *a: None)
    monkeypatch.setattr(tb, "_other_stream", lambda device, stream, *ts: recorded.extend(ts))
    inputs, outputs = call()
    held = {id(t) for t in recorded}
    assert all(id(t) in held for t in (*inputs, *outputs))
