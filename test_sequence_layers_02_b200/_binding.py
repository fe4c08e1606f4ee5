"""What the bindings of the operators around the scan share: the stream of a call, strides, checks.

Each of these operators runs on CUDA tensors only, on ``stream`` (default: the current stream of the
tensors' device), and returns without synchronising. Outputs and workspaces that a call makes itself
are allocated on that stream; inputs are marked as used by it where it is not the current one.
"""

from __future__ import annotations

import ctypes

import torch

from . import ttt_scan

_FLOATS = (torch.float32, torch.bfloat16)
TTTScanError = ttt_scan.TTTScanError


class Library:
    """The argument types of some functions of the library, set at the first call."""

    def __init__(self, functions: dict):
        self._functions = functions
        self._lib = None

    def __call__(self) -> ctypes.CDLL:
        if self._lib is None:
            lib = ttt_scan.lib()
            for name, (args, res) in self._functions.items():
                fn = getattr(lib, name)
                fn.argtypes, fn.restype = args, res
            self._lib = lib
        return self._lib


def check_device(name: str, x: torch.Tensor) -> torch.device:
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return x.device


def check_dtype(name: str, x: torch.Tensor) -> torch.dtype:
    if x.dtype not in _FLOATS:
        raise ValueError(f"{name}: expected float32 or bfloat16")
    return x.dtype


def check(name: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype, dev: torch.device) -> None:
    """Shape, type and device, and contiguous rows (the last dimension)."""
    if t.shape != shape or t.dtype != dtype or t.device != dev or \
            (t.stride(-1) != 1 and t.shape[-1] > 1):
        raise ValueError(f"{name}: expected {shape} {dtype} on {dev} with contiguous rows, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device} with strides {t.stride()}")


def check_whole(name: str, t, shape: tuple, dtype: torch.dtype, dev: torch.device):
    """As ``check`` for a tensor that has to be contiguous; its address, or None for None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {shape} {dtype} on {dev}, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device} with strides {t.stride()}")
    return t.data_ptr()


def out_dtype_of(out_dtype, default: torch.dtype) -> torch.dtype:
    if out_dtype is None:
        return default
    if out_dtype not in _FLOATS:
        raise ValueError("out_dtype: expected float32 or bfloat16")
    return out_dtype


def strides_of(*parts):
    """The strides of a call: None when every tensor is contiguous, else one array. A part is a
    tensor and the dimensions whose strides count, or a shape in the place of an absent tensor."""
    if all(not isinstance(t, torch.Tensor) or t.is_contiguous() for t, _ in parts):
        return None
    values = []
    for t, dims in parts:
        if isinstance(t, torch.Tensor):
            s = t.stride()
        else:
            s, step = [0] * len(t), 1
            for i in range(len(t) - 1, -1, -1):
                s[i] = step
                step *= t[i]
        values += [s[i] for i in dims]
    return (ctypes.c_longlong * len(values))(*values)


class On:
    """The stream of a call: ``with On(dev, stream, inputs) as s`` makes it the current one, for
    the allocations inside and for the device of the launch, and marks the inputs as used there."""

    __slots__ = ("dev", "stream", "inputs", "_ctx")

    def __init__(self, dev: torch.device, stream, inputs):
        self.dev, self.stream, self.inputs, self._ctx = dev, stream, inputs, None

    def __enter__(self):
        if self.stream is None and torch.cuda.current_device() == self.dev.index:
            return torch.cuda.current_stream(self.dev).cuda_stream
        s = self.stream if self.stream is not None else torch.cuda.current_stream(self.dev)
        if s.device != self.dev:
            raise ValueError(f"the stream is on {s.device}, the tensors on {self.dev}")
        if s != torch.cuda.current_stream(self.dev):
            for t in self.inputs:
                if t is not None:
                    t.record_stream(s)
        self._ctx = torch.cuda.stream(s)
        self._ctx.__enter__()
        return s.cuda_stream

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)
        return False


def raise_for(status: int, what: str) -> None:
    if status != ttt_scan.TTT_OK:
        raise TTTScanError(status, what)
