"""Short causal convolution (``include/ttt_conv.h``): the depthwise convolution over the last 2 to 4 tokens
that stands in front of a recurrence, on the queries and keys of ``ttt_scan.scan`` or on the input of
``ssm.selective_scan``.

    pre_t = bias + sum_j weight[:, j] x_{t - (K-1) + j},   y_t = SiLU(pre_t) (``silu``) or pre_t

Tensors are [B, T, D], or [B, H, T, d] with weight [H, d, K] and bias [H, d], the layout of the TTT
scan. A row of channels is contiguous; batch rows, heads and tokens may have any strides, so a
token-major projection can be given as ``x.unflatten(-1, (H, d)).transpose(1, 2)`` and comes out as
the contiguous [B, H, T, d] that ``ttt_scan.scan`` takes. CUDA tensors only; see ``_binding`` for
streams. There is no CPU fallback. Nothing is recorded for autograd: gradients come from
``causal_conv_backward``, called by hand.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._binding import (Library, On, check, check_float, check_whole, cuda_index, fit_ints, like,
                       out_dtype_of, raise_for, strides_of, workspace_of)
from .ttt_scan import IN_BF16, OUT_BF16

CONV_SILU = 1 << 16
CONV_PAD_ZERO = 1 << 20

_vp, _i, _u, _z = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_size_t
_lib = Library({
    "ttt_conv_forward": ([_vp] * 5 + [_i] * 5 + [_u] + [_vp] * 4, _i),
    "ttt_conv_backward_workspace_bytes": ([_i] * 5, _z),
    "ttt_conv_backward": ([_vp] * 5 + [_i] * 5 + [_u] + [_vp] * 8 + [_z, _vp], _i),
    "ttt_conv_step": ([_vp] * 5 + [_i] * 4 + [_u] + [_vp] * 3, _i),
})
_F32, _BF16 = torch.float32, torch.bfloat16
_OUTER = {3: (0, 0, 1), 4: (0, 1, 2)}  # dimensions of the strides between rows, heads, tokens


def _sizes(x, weight, bias, dev, tokens: bool):
    """B, H, T, d, K, the addresses of weight and bias; ``tokens``: x has a dimension of tokens."""
    shape = x.shape
    n = len(shape) + (0 if tokens else 1)
    if n == 3:
        H, channels = 1, (shape[-1],)
    elif n == 4:
        H, channels = shape[1], (shape[1], shape[-1])
    else:
        raise ValueError("x must be [B, T, D] or [B, H, T, d]" if tokens else
                         "x must be [B, D] or [B, H, d]")
    fit_ints("x", *shape)
    K = weight.shape[-1] if weight.dim() == len(channels) + 1 else 0
    w = check_whole("weight", weight, channels + (K,), _F32, dev)
    b = check_whole("bias", bias, channels, _F32, dev)
    return shape[0], H, shape[-2] if tokens else 1, shape[-1], K, w, b


def _mode(in_dtype, out_dtype, silu, pad_zero) -> int:
    return ((IN_BF16 if in_dtype is _BF16 else 0) | (OUT_BF16 if out_dtype is _BF16 else 0) |
            (CONV_SILU if silu else 0) | (CONV_PAD_ZERO if pad_zero else 0))


def causal_conv(x, weight, bias=None, *, silu: bool = False, state=None, lengths=None,
                out_dtype: Optional[torch.dtype] = None, y: Optional[torch.Tensor] = None,
                state_T: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None):
    """``(y, state_T) = causal_conv(x, weight, bias)`` over a prompt.

    x: [B, T, D] or [B, H, T, d], fp32 or bf16; weight: [D, K] or [H, d, K] fp32, K = 2, 3 or 4; bias: [D]
    or [H, d] fp32 or None; state: the K - 1 inputs before the first token, oldest first, [B, K-1, D] or
    [B, H, K-1, d] in x's type, or None for zeros; lengths: [B] int32 or None, the tokens of each row
    of a padded batch (those behind it are not read). y (``out_dtype``, default x's type) keeps its
    values behind a row's length; one made here is 0 there. state_T, the inputs before the next
    token, may be ``state`` itself.
    """
    dev, in_dtype = cuda_index("x", x), x.dtype
    B, H, T, d, K, w, b = _sizes(x, weight, bias, dev, True)
    xp = check("x", x, x.shape, in_dtype, dev)
    s_shape = x.shape[:-2] + (K - 1, d)
    sp = None if state is None else check("state", state, s_shape, in_dtype, dev)
    n = check_whole("lengths", lengths, (B,), torch.int32, dev)
    out_dtype = out_dtype_of(out_dtype, y, in_dtype)
    mode = _mode(in_dtype, out_dtype, silu, y is None)
    with On(dev, stream, (x, weight, bias, state, lengths, y, state_T)) as s:
        if y is None:
            y = like(x, out_dtype)
        yp = check("y", y, x.shape, out_dtype, dev)
        if state_T is None:
            state_T = (torch.empty(s_shape, dtype=in_dtype, device=dev) if state is None
                       else like(state, in_dtype))
        tp = check("state_T", state_T, s_shape, in_dtype, dev)
        o = _OUTER[x.dim()]
        st = strides_of(12, (x, o), (y, o), (s_shape if state is None else state, o), (state_T, o))
        rc = _lib.ttt_conv_forward(xp, w, b, sp, n, B, H, T, d, K, mode, st, yp, tp, s)
    raise_for(rc, "ttt_conv_forward")
    return y, state_T


def backward_workspace_bytes(B: int, H: int, T: int, d: int, K: int) -> int:
    """Bytes of device workspace ``ttt_conv_backward`` needs for these sizes."""
    return int(_lib.ttt_conv_backward_workspace_bytes(B, H, T, d, K))


def causal_conv_backward(x, weight, bias, dy, dstate_T=None, *, silu: bool = False, state=None,
                         lengths=None, workspace: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Gradients of ``<dy, y> + <dstate_T, state_T>`` for a ``causal_conv`` with the same arguments.

    dy: as y (fp32 or bf16); dstate_T: as state_T, contiguous, or None (zero). Returns dx and dstate
    (x's type; 0 behind a row's length), dweight and dbias (fp32, dbias None without a bias).
    ``workspace`` (optional): at least ``backward_workspace_bytes`` bytes, not shared by calls that
    overlap.
    """
    dev, in_dtype = cuda_index("x", x), x.dtype
    B, H, T, d, K, w, b = _sizes(x, weight, bias, dev, True)
    xp = check("x", x, x.shape, in_dtype, dev)
    gp = check_float("dy", dy, x.shape, dev)
    s_shape = x.shape[:-2] + (K - 1, d)
    sp = None if state is None else check("state", state, s_shape, in_dtype, dev)
    ds_T = check_whole("dstate_T", dstate_T, s_shape, in_dtype, dev)
    n = check_whole("lengths", lengths, (B,), torch.int32, dev)
    o = _OUTER[x.dim()]
    st = strides_of(9, (x, o), (dy, o), (s_shape if state is None else state, o))
    with On(dev, stream, (x, weight, bias, dy, dstate_T, state, lengths, workspace)) as s:
        workspace, wp, wn = workspace_of(workspace, backward_workspace_bytes(B, H, T, d, K), dev)
        dx = like(x, in_dtype)
        dstate = torch.empty(s_shape, dtype=in_dtype, device=dev)
        dweight = torch.empty_like(weight)
        dbias = None if bias is None else torch.empty_like(bias)
        rc = _lib.ttt_conv_backward(xp, w, b, sp, n, B, H, T, d, K,
                                    _mode(in_dtype, dy.dtype, silu, False), st, gp, ds_T,
                                    dx.data_ptr(), dweight.data_ptr(),
                                    None if bias is None else dbias.data_ptr(), dstate.data_ptr(),
                                    wp, wn, s)
    raise_for(rc, "ttt_conv_backward")
    return dict(dx=dx, dweight=dweight, dbias=dbias, dstate=dstate)


def causal_conv_step(x, weight, bias, state, *, silu: bool = False, active=None,
                     out_dtype: Optional[torch.dtype] = None, y: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None):
    """``y = causal_conv_step(x, weight, bias, state)``: one token of every row.

    x: [B, D] or [B, H, d]; state: [B, K-1, D] or [B, H, K-1, d] in x's type, moved on by one token IN
    PLACE; active: [B] uint8 or None, 0 = the row's state and y are left as they were (a y made here
    is 0 there). A chain of steps equals ``causal_conv``.
    """
    dev, in_dtype = cuda_index("x", x), x.dtype
    B, H, _, d, K, w, b = _sizes(x, weight, bias, dev, False)
    xp = check("x", x, x.shape, in_dtype, dev)
    sp = check("state", state, x.shape[:-1] + (K - 1, d), in_dtype, dev)
    a = check_whole("active", active, (B,), torch.uint8, dev)
    out_dtype = out_dtype_of(out_dtype, y, in_dtype)
    mode = _mode(in_dtype, out_dtype, silu, y is None)
    with On(dev, stream, (x, weight, bias, state, active, y)) as s:
        if y is None:
            y = like(x, out_dtype)
        yp = check("y", y, x.shape, out_dtype, dev)
        o = (0, 1) if x.dim() == 3 else (0, 0)
        st = strides_of(7, (x, o), (y, o), (state, _OUTER[state.dim()]))
        rc = _lib.ttt_conv_step(xp, w, b, sp, a, B, H, d, K, mode, st, yp, s)
    raise_for(rc, "ttt_conv_step")
    return y
