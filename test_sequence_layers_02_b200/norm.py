"""Root-mean-square norm between two blocks (``include/ttt_norm.h``):

    s = x + residual,   y = s / sqrt(mean(s^2) + eps) * weight

with y in fp32 or bf16 (``rmsnorm``, and ``rmsnorm_backward`` for training) or in 8 bits with scales for the
projections behind it (``rmsnorm_fp8``). Rows are the last dimension; they are contiguous, and a
2-D tensor may have any row stride from D up (rows of an expanded tensor have to be copied first). CUDA
tensors only; see ``_binding`` for streams. There is no CPU fallback. Nothing is recorded for
autograd: gradients come from ``rmsnorm_backward``, called by hand.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._binding import (Library, On, check, check_float, check_whole, cuda_index, fit_ints, like,
                       out_dtype_of, raise_for, workspace_of, arrays)
from .ttt_scan import IN_BF16, OUT_BF16

NORM_SUM_BF16 = 1 << 18
NORM_Y_E4M3 = 1 << 19

_vp, _i, _u, _f, _z = (ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_float,
                       ctypes.c_size_t)
_lib = Library({
    "ttt_norm_forward": ([_vp] * 3 + [_i, _i, _f, _u, _i] + [_vp] * 5, _i),
    "ttt_norm_backward_workspace_bytes": ([_i, _i], _z),
    "ttt_norm_backward": ([_vp] * 4 + [_i, _i, _f, _u] + [_vp] * 4 + [_z, _vp], _i),
})


_F32, _BF16 = torch.float32, torch.bfloat16


def _rows(name, t, shape, dtype, dev):
    """The address and the row stride of a tensor of this shape, after its checks."""
    p = check(name, t, shape, dtype, dev)
    if t.is_contiguous():
        return p, shape[-1]
    if len(shape) != 2:
        raise ValueError(f"{name}: expected contiguous {tuple(shape)} (2-D tensors may have strides)")
    return p, t.stride(0) if shape[0] > 1 else shape[-1]


def _strides(D, *lds):
    for v in lds:
        if v != D:
            return arrays[4](*lds)
    return None


def _shape(name, t):
    """M, D of a tensor of rows."""
    shape = t.shape
    if not shape:
        raise ValueError(f"{name} must be [..., D]")
    D = shape[-1]
    M = t.numel() // D if D else 0
    fit_ints(name, M, D)
    return shape, M, D


def _forward(x, weight, residual, eps, mode, group, y, y_dtype, s, stream):
    dev, dtype = cuda_index("x", x), x.dtype
    shape, M, D = _shape("x", x)
    w = check_whole("weight", weight, (D,), _F32, dev)
    xp, ld_x = _rows("x", x, shape, dtype, dev)
    rp, ld_r, sp, ld_s, sum_dtype = None, D, None, D, dtype
    if residual is not None:
        sum_dtype = residual.dtype
        cuda_index("residual", residual)
        rp, ld_r = _rows("residual", residual, shape, sum_dtype, dev)
    elif s is not None:
        raise ValueError("s: there is none without a residual (it would be x)")
    mode |= ((IN_BF16 if dtype is _BF16 else 0) | (NORM_SUM_BF16 if sum_dtype is _BF16 else 0))
    scale = None
    with On(dev, stream, (x, weight, residual, y, s)) as st:
        if y is None:
            y = like(x, y_dtype)
        yp, ld_y = _rows("y", y, shape, y_dtype, dev)
        if residual is not None:
            if s is None:
                s = like(residual, sum_dtype)
            sp, ld_s = _rows("s", s, shape, sum_dtype, dev)
        if mode & NORM_Y_E4M3:
            n = -(-D // 128) if group else 1
            scale = weight.new_empty((*shape[:-1], n))
        rc = _lib.ttt_norm_forward(xp, rp, w, M, D, eps, mode, group,
                                   _strides(D, ld_x, ld_r, ld_y, ld_s), yp, sp,
                                   None if scale is None else scale.data_ptr(), st)
    raise_for(rc, "ttt_norm_forward")
    return y, scale, x if residual is None else s


def rmsnorm(x, weight, residual=None, *, eps: float = 1e-6, out_dtype: Optional[torch.dtype] = None,
            y: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None):
    """``(y, s) = rmsnorm(x, weight, residual)``.

    x: [..., D] fp32 or bf16, D up to 16384; weight: [D] fp32; residual: [..., D] fp32 or bf16 (its own
    type) or None. y: ``out_dtype``, default x's type, of the unrounded sum; s: the sum in the
    residual's type, or x itself without a residual. ``s`` may be given as the residual (or as x, where the
    types agree) to update the residual stream in place.
    """
    out_dtype = out_dtype_of(out_dtype, y, x.dtype)
    mode = OUT_BF16 if out_dtype is _BF16 else 0
    y, _, s = _forward(x, weight, residual, eps, mode, 0, y, out_dtype, s, stream)
    return y, s


def rmsnorm_fp8(x, weight, residual=None, *, eps: float = 1e-6, group: int = 0,
                y: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None):
    """``(y, scale, s) = rmsnorm_fp8(x, weight, residual)``: y as float8_e4m3fn codes.

    scale: fp32 [..., 1], the row's max |y| / 448 (``group=0``), or [..., ceil(D / 128)], that of each 128
    columns (``group=128``); the value of a code is code * scale, and a code is that of the fp32 quotient y / scale. A
    row or group with a NaN has NaN for its scale and codes. Otherwise as ``rmsnorm``.
    """
    if group not in (0, 128):
        raise ValueError("group: expected 0 (a scale per row) or 128")
    return _forward(x, weight, residual, eps, NORM_Y_E4M3, group, y, torch.float8_e4m3fn, s, stream)


def backward_workspace_bytes(M: int, D: int) -> int:
    """Bytes of device workspace ``ttt_norm_backward`` needs for M rows."""
    return int(_lib.ttt_norm_backward_workspace_bytes(M, D))


def rmsnorm_backward(dy, s, weight, ds=None, *, eps: float = 1e-6,
                     dx: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Gradients of ``<dy, y> + <ds, s>`` for ``(y, s) = rmsnorm(x, weight, residual)``.

    dy: [..., D] fp32 or bf16; s: as ``rmsnorm`` returned it (the gradient is taken at these, rounded
    values); ds: the gradient that reaches s from elsewhere, s's type, or None. Returns dx, the gradient
    of x and of the residual alike (s's type; may be given as ``ds`` itself), and dweight (fp32).
    ``workspace`` (optional): at least ``backward_workspace_bytes`` bytes, not shared by calls that
    overlap.
    """
    dev, dtype = cuda_index("s", s), s.dtype
    shape, M, D = _shape("s", s)
    w = check_whole("weight", weight, (D,), _F32, dev)
    sp, ld_s = _rows("s", s, shape, dtype, dev)
    check_float("dy", dy, shape, dev)
    gp, ld_g = _rows("dy", dy, shape, dy.dtype, dev)
    ep, ld_e = (None, D) if ds is None else _rows("ds", ds, shape, dtype, dev)
    mode = (OUT_BF16 if dy.dtype is _BF16 else 0) | (NORM_SUM_BF16 if dtype is _BF16 else 0)
    with On(dev, stream, (dy, s, weight, ds, dx, workspace)) as st:
        if dx is None:
            dx = like(s, dtype)
        op, ld_o = _rows("dx", dx, shape, dtype, dev)
        workspace, wp, wn = workspace_of(workspace, backward_workspace_bytes(M, D), dev)
        dweight = torch.empty_like(weight)
        rc = _lib.ttt_norm_backward(gp, sp, w, ep, M, D, eps, mode,
                                    _strides(D, ld_g, ld_s, ld_e, ld_o), op, dweight.data_ptr(), wp,
                                    wn, st)
    raise_for(rc, "ttt_norm_backward")
    return dict(dx=dx, dweight=dweight)
