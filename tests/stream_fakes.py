"""Stand-ins for torch's streams, so that a machine without a GPU can see on
which stream a call allocates and which tensors it records where."""
import contextlib

import torch

from dequantize_reduce_transfer_amd import layer


class FakeStream:
    def __init__(self, name, handle, device):
        self.name, self.cuda_stream, self.device = name, handle, device


class LoggedTensor(torch.Tensor):
    """A CPU tensor that passes for one on a GPU and keeps the streams it is
    recorded on."""

    is_cuda = property(lambda self: True)

    def record_stream(self, stream):
        self.__dict__.setdefault("recorded", []).append(stream.name)


def logged(*shape, dtype=torch.uint8):
    return torch.zeros(*shape, dtype=dtype).as_subclass(LoggedTensor)


def recorded(t):
    return set(t.__dict__.get("recorded", []))


class FakeStreams:
    """Patches torch.cuda's current stream; ``now`` is the current one."""

    def __init__(self, monkeypatch):
        device = torch.device("cpu")
        self.caller, self.named = FakeStream("caller", 1, device), FakeStream("named", 2, device)
        self.now = self.caller
        monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: self.now)
        monkeypatch.setattr(layer, "_raw_stream", lambda index: self.now.cuda_stream)
        monkeypatch.setattr(torch.cuda, "set_stream", self._set)
        monkeypatch.setattr(torch.cuda, "stream", self._current)
        monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())

    def _set(self, stream):
        self.now = stream

    @contextlib.contextmanager
    def _current(self, stream):
        before, self.now = self.now, stream
        try:
            yield
        finally:
            self.now = before
