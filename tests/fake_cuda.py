"""Host tensors that pass the binding's checks for device tensors, and a
library that records its calls and launches nothing: what the binding
allocates, on which stream and with which pointers, shown without a GPU."""

import contextlib

import torch


class FakeCuda(torch.Tensor):
    is_cuda = True


def fake(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(FakeCuda)


class FakeStream:
    cuda_stream = 0x51


class FakeLibrary:
    """Every entry succeeds; cross_attention_workspace asks for `floats`."""

    def __init__(self, floats=64):
        self.calls, self.floats = [], floats

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            if name == "cross_attention_workspace":
                args[1]._obj.value = self.floats
            return 0
        return call


class Recorder:
    """Patches the binding; `allocations` holds (shape, stream current then)."""

    def __init__(self, monkeypatch, binding, floats=64):
        self.current, self.allocations = None, []
        self.library = FakeLibrary(floats)
        plain_empty = torch.empty

        @contextlib.contextmanager
        def stream_context(stream):
            before, self.current = self.current, stream
            yield
            self.current = before

        def empty(*args, **kw):
            t = plain_empty(*args, **kw).as_subclass(FakeCuda)
            self.allocations.append((tuple(t.shape), self.current))
            return t

        monkeypatch.setattr(binding, "lib", lambda: self.library)
        monkeypatch.setattr(binding, "_raw_stream", lambda stream, *_: 0 if stream is None else stream.cuda_stream)
        monkeypatch.setattr(binding, "_stream", lambda stream: 0 if stream is None else stream.cuda_stream)
        monkeypatch.setattr(torch.cuda, "stream", stream_context)
        monkeypatch.setattr(torch, "empty", empty)
        monkeypatch.setattr(torch, "empty_like", lambda t: empty(t.shape, dtype=t.dtype))
