"""Tensors that the binding allocates come from the stream that their call runs on."""
from contextlib import contextmanager

import pytest
import torch


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


class FakeTensor:
    device = torch.device("cuda", 0)

    def __init__(self, handle):
        self.allocated_on, self.recorded = handle, []

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


@pytest.fixture
def fake_cuda(monkeypatch, native_lib):
    """torch.empty notes the current stream (7 at first; the default stream is 0)."""
    current = [FakeStream(7)]

    @contextmanager
    def on(stream):
        before = current[0]
        current[0] = stream
        yield
        current[0] = before

    def set_stream(stream):
        current[0] = stream

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[0])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: FakeStream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(handle))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "set_stream", set_stream)
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: FakeTensor(current[0].cuda_stream))
    monkeypatch.setattr(native_lib, "_raw_stream", None)
    return native_lib


@pytest.mark.parametrize("as_stream", [False, True])
@pytest.mark.parametrize("handle", [None, 7, 0, 1, 2, 4096])
def test_blocks_come_from_the_calls_stream(fake_cuda, handle, as_stream):
    want = {None: 7, 1: 0}.get(handle, handle)
    if as_stream:
        handle = FakeStream(want)
    out = fake_cuda._output(None, "Y", 4, 8, 0, handle)
    scratch = fake_cuda._scratch(None, 0, handle, lambda *shape: 64, 4, 8)
    assert out.allocated_on == want and scratch.allocated_on == want
    # an output read on the current stream is not handed out again before that is done
    assert out.recorded == ([] if want == 7 else [7])
    assert scratch.recorded == []
    assert torch.cuda.current_stream().cuda_stream == 7
