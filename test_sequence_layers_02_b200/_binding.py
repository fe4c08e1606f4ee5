"""What the bindings of the operators around the scan share: the stream of a call, strides, checks.

Each of these operators runs on CUDA tensors only, on ``stream`` (default: the current stream of the
tensors' device), and returns without synchronising. Outputs and workspaces that a call makes itself
are allocated on that stream; inputs are marked as used by it where it is not the current one.

The calls are outside autograd, as ``ttt_scan``'s are: their outputs carry no ``grad_fn``, also for inputs that
require a gradient, and gradients come from the ``*_backward`` calls, made by hand (or from a
``torch.autograd.Function`` of the caller's around both).

A one-token step takes the GPU a few microseconds, so these checks are written for few and cheap
calls into torch: a tensor's device by its number, contiguity before strides.
"""

from __future__ import annotations

import ctypes

import torch

from . import ttt_scan

FLOATS = (torch.float32, torch.bfloat16)
TTTScanError = ttt_scan.TTTScanError
_F32 = torch.float32


class Library:
    """Some functions of the library with their argument types, looked up at the first use."""

    def __init__(self, functions: dict):
        self._functions = functions

    def __getattr__(self, name):
        if name not in self._functions:
            raise AttributeError(name)
        args, res = self._functions[name]
        fn = getattr(ttt_scan.lib(), name)
        fn.argtypes, fn.restype = args, res
        setattr(self, name, fn)
        return fn


def cuda_index(name: str, x: torch.Tensor) -> int:
    """The CUDA device of x, by number; its type is float32 or bfloat16."""
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dtype not in FLOATS:
        raise ValueError(f"{name}: expected float32 or bfloat16")
    return x.get_device()


def fit_ints(name: str, *sizes) -> None:
    """The sizes of a call are C ints, to which ctypes would cut larger ones without a word."""
    if max(sizes) > 0x7fffffff:
        raise ValueError(f"{name}: sizes up to 2147483647, got {tuple(sizes)}")


def _refuse(name, t, shape, dtype, dev, what):
    raise ValueError(f"{name}: expected {what} {tuple(shape)} {dtype} on cuda:{dev}, got "
                     f"{tuple(t.shape)} {t.dtype} on {t.device} with strides {t.stride()}")


def check(name: str, t: torch.Tensor, shape, dtype: torch.dtype, dev: int) -> int:
    """Shape, type and device, and contiguous rows (the last dimension); the tensor's address."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or \
            not (t.is_contiguous() or t.stride(-1) == 1 or t.shape[-1] <= 1):
        _refuse(name, t, shape, dtype, dev, "rows of")
    return t.data_ptr()


def check_float(name: str, t: torch.Tensor, shape, dev: int) -> int:
    """As ``check``, of either floating type."""
    if t.dtype not in FLOATS:
        raise ValueError(f"{name}: expected float32 or bfloat16")
    return check(name, t, shape, t.dtype, dev)


def check_whole(name: str, t, shape, dtype: torch.dtype, dev: int):
    """As ``check`` for a tensor that has to be contiguous; None for None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _refuse(name, t, shape, dtype, dev, "contiguous")
    return t.data_ptr()


def out_dtype_of(out_dtype, y, default: torch.dtype) -> torch.dtype:
    """The type of an output: of the given tensor, as asked for, or the default."""
    if y is not None:
        out_dtype = y.dtype
    elif out_dtype is None:
        return default
    if out_dtype not in FLOATS:
        raise ValueError("out_dtype: expected float32 or bfloat16")
    return out_dtype


def like(x: torch.Tensor, dtype: torch.dtype) -> torch.Tensor:
    """A contiguous tensor of x's shape and device, not initialised (``empty_like``, where it gives
    that, takes a third of ``empty``'s time)."""
    if not x.is_contiguous():
        return torch.empty(x.shape, dtype=dtype, device=x.device)
    return torch.empty_like(x) if x.dtype is dtype else torch.empty_like(x, dtype=dtype)


def _contiguous_strides(shape):
    s, step = [], 1
    for n in reversed(shape):
        s.append(step)
        step *= n
    return s[::-1]


arrays = {n: ctypes.c_longlong * n for n in (4, 7, 8, 9, 12, 14)}


def strides_of(count: int, *parts):
    """The strides of a call: None when every tensor is contiguous, else an array of ``count``. A part
    is a tensor and the dimensions whose strides count, or a shape in the place of an absent tensor."""
    for t, _ in parts:
        if isinstance(t, torch.Tensor) and not t.is_contiguous():
            break
    else:
        return None
    values = []
    for t, dims in parts:
        s = t.stride() if isinstance(t, torch.Tensor) else _contiguous_strides(t)
        for i in dims:
            values.append(s[i])
    return arrays[count](*values)


# Torch's private calls, without the public ones' work around them; a release that lacks them has those.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())
_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None) or
               (lambda dev: torch.cuda.current_stream(dev).cuda_stream))


class On:
    """The stream of a call: ``with On(dev, stream, inputs) as s`` makes it the current one, for
    the allocations inside and for the device of the launch, and marks the inputs as used there."""

    __slots__ = ("dev", "stream", "inputs", "ctx")

    def __init__(self, dev: int, stream, inputs):
        self.dev, self.stream, self.inputs, self.ctx = dev, stream, inputs, None

    def __enter__(self) -> int:
        if self.stream is None and _current_device() == self.dev:
            return _raw_stream(self.dev)
        now = torch.cuda.current_stream(self.dev)
        s = now if self.stream is None else self.stream
        if s.device.index != self.dev:
            raise ValueError(f"the stream is on {s.device}, the tensors on cuda:{self.dev}")
        if s != now:
            for t in self.inputs:
                if t is not None:
                    t.record_stream(s)
        self.ctx = torch.cuda.stream(s)
        self.ctx.__enter__()
        return s.cuda_stream

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def workspace_of(workspace, need: int, dev: int):
    """A call's workspace (allocated here when None), its address and its bytes."""
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on cuda:{dev}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def raise_for(status: int, what: str) -> None:
    if status != 0:
        raise TTTScanError(status, what)
