"""What the binding's calls use of torch.cuda and of the library, replaced for
tests without a GPU: streams with handles, a record of every allocation with
the stream that was current for it, and launches that are only recorded."""
import contextlib
import threading

import torch

import boolean_weight_amd as bw


class Stream:
    def __init__(self, handle, device=0):
        self.cuda_stream, self.device = handle, device


class DeviceTensor(torch.Tensor):
    """A host tensor that says it is on device 0."""

    def get_device(self):
        return 0

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", 0)


def on_device(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(DeviceTensor)


class Gpu:
    POOL = 0x9000  # what an external stream of handle 0 is: one of torch's own

    def __init__(self, monkeypatch, launch=None):
        self.local, self.allocated, self.launched = threading.local(), [], []
        self.capturing = set()  # handles of streams that are being captured
        real, lib, empty = bw.load_library(), self, torch.empty

        class Library:
            def __getattr__(self, name):
                if name.endswith(("_bytes", "_init", "_stack")):
                    return getattr(real, name)

                def call(*args):
                    lib.launched.append((name, args))
                    if launch:
                        launch(name, args)
                    return 0
                return call

        def alloc(size, dtype=torch.float32, device=None):
            if device is None or torch.device(device).type != "cuda":
                return empty(size, dtype=dtype, device=device)
            t = empty(size, dtype=dtype).as_subclass(DeviceTensor)
            self.allocated.append((self.current().cuda_stream, t))
            return t

        @contextlib.contextmanager
        def use(stream):
            self.stack().append(stream)
            try:
                yield
            finally:
                self.stack().pop()

        library = Library()
        cuda = torch.cuda
        monkeypatch.setattr(bw, "load_library", lambda: library)
        monkeypatch.setattr(bw, "_WORKSPACES", {})
        monkeypatch.setattr(bw, "_WORKSPACE_LOCKS", {})
        monkeypatch.setattr(bw, "_raw_stream", lambda dev: self.current().cuda_stream)
        monkeypatch.setattr(bw, "_current_device", lambda: 0)
        monkeypatch.setattr(torch, "empty", alloc)
        monkeypatch.setattr(cuda, "Stream", Stream)
        monkeypatch.setattr(cuda, "ExternalStream",
                            lambda handle, device=None: Stream(handle or self.POOL))
        monkeypatch.setattr(cuda, "current_stream", lambda device=None: self.current())
        monkeypatch.setattr(cuda, "default_stream", lambda device=None: Stream(0))
        monkeypatch.setattr(cuda, "current_device", lambda: 0)
        monkeypatch.setattr(cuda, "stream", use)
        monkeypatch.setattr(cuda, "device", lambda dev: contextlib.nullcontext())
        monkeypatch.setattr(cuda, "is_current_stream_capturing",
                            lambda: self.current().cuda_stream in self.capturing)
        self.use = use

    def stack(self):
        if not hasattr(self.local, "stack"):
            self.local.stack = [Stream(0)]
        return self.local.stack

    def current(self):
        return self.stack()[-1]
