"""Stand-ins for torch's CUDA side and for the library, which record on which stream
memory is taken and what every entry point is called with.  No device needed."""
import contextlib
import itertools

import torch

_addresses = itertools.count(4096, 4096)


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Tensor:
    is_cuda = True
    device = torch.device("cuda", 0)

    def __init__(self, shape, dtype, home=None):
        self.shape, self.dtype, self.home = tuple(shape), dtype, home
        self.address, self.used_on = next(_addresses), set()

    def is_contiguous(self):
        return True

    def numel(self):
        n = 1
        for d in self.shape:
            n *= d
        return n

    def data_ptr(self):
        return self.address

    def record_stream(self, stream):
        self.used_on.add(stream.cuda_stream)


class Torch:
    """What experts.py takes from the torch module; `current` is the current stream."""
    float16, float32, int32, uint8 = torch.float16, torch.float32, torch.int32, torch.uint8

    def __init__(self):
        self.current = Stream(1)
        self.cuda = self._C = self

    def empty(self, shape, dtype, device):
        return Tensor(shape if isinstance(shape, tuple) else (shape,), dtype,
                      self.current.cuda_stream)

    @contextlib.contextmanager
    def stream(self, stream):
        before, self.current = self.current, stream
        yield
        self.current = before

    def current_stream(self, device=None):
        return self.current

    def _cuda_getDevice(self):
        return 0

    def _cuda_getCurrentRawStream(self, index):
        return self.current.cuda_stream


class Library:
    """Every entry point succeeds; `calls` holds (name, arguments)."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            # a plan: no number, so that the library itself can never take it for one
            return object() if "create" in name else 0
        return call


def install(monkeypatch):
    """experts.py on the stand-ins: (torch, library)."""
    from tma_pipelined_tensor_fp16_gb300 import experts
    fake, library = Torch(), Library()
    monkeypatch.setitem(experts._modules, "torch", fake)
    monkeypatch.setattr(experts, "lib", lambda: library)
    return fake, library
