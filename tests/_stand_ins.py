"""Stand-ins for CUDA tensors, torch and the library, so that what the layer
calls do around their launches can be tested without a GPU, through the
extension and through the interpreter."""
import contextlib
import ctypes
import importlib.machinery
import importlib.util
import itertools
import os
import shutil
import types
import weakref

import torch

from dense_fp32_tiled_gb300 import _layers
from dense_fp32_tiled_gb300 import build as sg_build

_addresses = itertools.count(1)


class Tensor:
    """Shape, strides, type and an address of a tensor on GPU 0; no memory."""

    def __init__(self, shape, dtype=torch.bfloat16, strides=None, address=None):
        self.shape, self.dtype, self.device, self.is_cuda = torch.Size(shape), dtype, torch.device("cuda:0"), True
        if strides is None:
            strides, n = [], 1
            for s in reversed(shape):
                strides.insert(0, n)
                n *= max(s, 1)
        self._strides = tuple(strides)
        self._address = next(_addresses) << 32 if address is None else address  # far apart, aligned

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self._strides

    def is_contiguous(self):
        return self._strides == Tensor(self.shape)._strides

    def data_ptr(self):
        return self._address

    def get_device(self):
        return 0

    def numel(self):
        return self.shape.numel()

    def transpose(self, a, b):
        shape, strides = list(self.shape), list(self._strides)
        shape[a], shape[b], strides[a], strides[b] = shape[b], shape[a], strides[b], strides[a]
        return Tensor(shape, self.dtype, strides, self._address)


class Stream:
    def __init__(self, index=0):
        self.device = types.SimpleNamespace(index=index)


def fast_call(directory):
    """A copy of the extension with a binding of its own (the loaded one keeps its)."""
    sg_build.build_fast_call()
    path = os.path.join(directory, "_fast_call.so")
    shutil.copy(sg_build.FAST_CALL, path)
    spec = importlib.util.spec_from_loader("_fast_call", importlib.machinery.ExtensionFileLoader("_fast_call", path))
    return importlib.util.module_from_spec(spec)


NAMES = [f for op in ("linear_forward", "linear_backward", "expert_linear_forward", "expert_linear_backward", "expert_sort")
         for f in (op, op + "_workspace_size")] + ["expert_gather", "expert_combine", "expert_combine_backward"]


class Library:
    """The library's functions, each an attribute that a test sets; `calls` counts those that were made."""

    def __init__(self, real):
        self.calls, self.callbacks, self.does = 0, {}, {}
        for name in NAMES:
            fn = getattr(real, name)

            def call(*args, name=name):
                if name.endswith("_workspace_size"):
                    return self.does.get(name, lambda *a: 0)(*args)
                self.calls += 1
                return self.does.get(name, lambda *a: 0)(*args)

            self.callbacks[name] = ctypes.CFUNCTYPE(fn.restype, *fn.argtypes)(call)
            setattr(self, name, self.callbacks[name])  # arguments are converted as the real one's are

    def addresses(self):
        return {n: ctypes.cast(c, ctypes.c_void_p).value for n, c in self.callbacks.items()}


def install(monkeypatch, real, way, directory, addresses=None):
    """Puts stand-ins in the place of torch and of the library for the calls of _layers."""
    lib, made = Library(real), []

    def empty(shape, dtype=None, device=None):
        t = Tensor((shape,) if isinstance(shape, int) else tuple(shape), dtype)
        made.append(weakref.ref(t))
        return t

    @contextlib.contextmanager
    def on(which):
        lib.entered.append(which)
        yield

    lib.made, lib.entered = made, []
    names = {n: getattr(torch, n) for n in ("float32", "bfloat16", "float16", "int32", "int64", "uint8")}
    stand_in = types.SimpleNamespace(empty=empty, Tensor=Tensor, cuda=types.SimpleNamespace(
        current_device=lambda: 0, stream=on, device=on), **names)
    monkeypatch.setattr(_layers, "torch", stand_in)
    monkeypatch.setattr(_layers, "_lib", lib)
    monkeypatch.setattr(_layers, "_types", {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
    monkeypatch.setattr(_layers, "_raw_stream", lambda device: 77)
    fast = None
    if way == "extension":
        fast = fast_call(directory)
        fast.bind({**lib.addresses(), **(addresses or {})},
                  _layers.bound(stand_in, lambda device: 77, lambda: 0))
    monkeypatch.setattr(_layers, "_fast", fast)
    return lib
