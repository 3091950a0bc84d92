"""A stand-in for the CUDA side of the bindings, for tests of what the wrappers
pass and allocate without a GPU: CPU tensors that say they lie on device 0,
streams that only have a handle, and a library whose calls are recorded."""
import contextlib

import torch

from paged_kv_attention_decode_gb300 import _binding

WORKSPACE_BYTES = 4096


class OnDevice(torch.Tensor):
    """A CPU tensor that says it lies on CUDA device 0."""

    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.__dict__.setdefault("recorded", []).append(stream.cuda_stream)


def dev(t):
    return t.as_subclass(OnDevice)


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class StandIn:
    """`calls`: (name, arguments) of every library call; `made`: (address, bytes,
    handle of the stream that was current) of every tensor the wrappers made."""

    def __init__(self, monkeypatch):
        self.calls, self.made, self.now = [], [], Stream(0)
        mp = monkeypatch

        @contextlib.contextmanager
        def stream(s):
            before, self.now = self.now, s
            try:
                yield
            finally:
                self.now = before

        def noted(make):
            def f(*a, **kw):
                t = dev(make(*a, **kw))
                self.made.append((t.data_ptr(), t.numel() * t.element_size(), self.now.cuda_stream))
                return t
            return f

        mp.setattr(_binding, "_lib", self)
        mp.setattr(_binding, "_cuda_device", lambda: 0)
        mp.setattr(_binding, "_raw_stream", lambda d: self.now.cuda_stream)
        mp.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: self.now.cuda_stream, raising=False)
        mp.setattr(torch.cuda, "current_device", lambda: 0)
        mp.setattr(torch.cuda, "current_stream", lambda *a: self.now)
        mp.setattr(torch.cuda, "default_stream", lambda *a: Stream(0))
        mp.setattr(torch.cuda, "ExternalStream", Stream)
        mp.setattr(torch.cuda, "stream", stream)
        mp.setattr(torch, "empty", noted(torch.empty))
        mp.setattr(torch, "empty_like", noted(torch.empty_like))

    def __getattr__(self, name):
        if not name.startswith("pa_"):
            raise AttributeError(name)

        def call(*args):
            if name.endswith("_bytes"):
                return WORKSPACE_BYTES
            if name == "pa_decode_partition_for":
                return 512
            self.calls.append((name, args))
            return 0
        return call
