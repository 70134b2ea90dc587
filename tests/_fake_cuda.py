"""A CUDA of several devices and streams that is not there: tensors that say
they lie on a device, the current device and stream, and a library whose calls
are written down. For tests of what the binding makes where; nothing runs."""
import contextlib

import torch


class Tensor(torch.Tensor):
    """CPU memory that claims to lie on CUDA device ``index``, made on ``pool``."""

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        if func is torch.Tensor.get_device:
            return args[0].index
        if func == torch.Tensor.is_cuda.__get__:
            return True
        if func == torch.Tensor.device.__get__:
            return torch.device("cuda", args[0].index)
        with torch._C.DisableTorchFunctionSubclass():
            r = func(*args, **(kwargs or {}))
        if isinstance(r, torch.Tensor):
            return dress(r, args[0].index, args[0].pool, args[0].users)
        return r

    def record_stream(self, stream):
        self.users.append(stream)


def dress(t, index, pool, users=None):
    t = t.as_subclass(Tensor)
    t.index, t.pool, t.users = index, pool, [] if users is None else users
    return t


class Stream:
    def __init__(self, index, handle):
        self.device = torch.device("cuda", index)
        self.device_index = index
        self.cuda_stream = handle


class Library:
    """Every call is noted as (name, current device, arguments) and succeeds;
    sizes of workspaces are 64 bytes."""

    def __init__(self, cuda):
        self.cuda, self.calls = cuda, []

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return lambda *a: 64

        def call(*args):
            self.calls.append((name, self.cuda.device, args))
            return 0
        return call


class Cuda:
    """Current device and its current stream; the default stream's handle is 0
    on every device."""

    def __init__(self, monkeypatch, module, devices=2):
        self.device = 0
        self.streams = [Stream(i, 0) for i in range(devices)]
        self.made = []
        self.lib = Library(self)
        real_empty = torch.empty

        def empty(*shape, dtype=None, device=None):
            where = torch.device("cpu" if device is None else device)
            t = real_empty(*shape, dtype=dtype)
            if where.type != "cuda":
                return t
            index = self.device if where.index is None else where.index
            t = dress(t, index, self.streams[index])
            self.made.append(t)
            return t

        @contextlib.contextmanager
        def on_stream(stream):
            i, old, was = stream.device_index, self.streams[stream.device_index], self.device
            self.device, self.streams[i] = i, stream
            try:
                yield
            finally:
                self.device, self.streams[i] = was, old

        @contextlib.contextmanager
        def on_device(index):
            was, self.device = self.device, index
            try:
                yield
            finally:
                self.device = was

        def current(index=None):
            return self.streams[self.device if index is None else index]

        for name, f in (("stream", on_stream), ("device", on_device), ("current_stream", current),
                        ("current_device", lambda: self.device), ("device_count", lambda: devices)):
            monkeypatch.setattr(torch.cuda, name, f)
        monkeypatch.setattr(torch, "empty", empty)
        monkeypatch.setattr(module, "_raw_stream", lambda i: self.streams[i].cuda_stream)
        monkeypatch.setattr(module, "load_library", lambda: self.lib)
        monkeypatch.setattr(module, "_devices", None, raising=False)

    def tensor(self, shape, dtype, index=0):
        return dress(torch.zeros(shape, dtype=dtype), index, self.streams[index])
