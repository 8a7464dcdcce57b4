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
