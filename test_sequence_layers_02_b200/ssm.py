"""Selective state space scan (``include/ttt_ssm.h``), a sibling of the TTT scan whose state is N numbers for
each channel:

    dt_t = softplus(delta_t + delta_bias)
    h_t  = exp(dt_t A) h_{t-1} + dt_t u_t Bm_t,   y_t = (Cm_t . h_t + D u_t) SiLU(z_t)

for prompts (``selective_scan``), training (``selective_scan_backward``) and single tokens
(``selective_step``). u, delta, z, y are [B, T, D], Bm and Cm [B, T, G, N] (or [B, T, N] for one
group), fp32 or bf16, with contiguous rows and any strides between batch rows, tokens and groups;
parameters and states are fp32. CUDA tensors only; see ``_binding`` for streams. There is no CPU
fallback. Nothing is recorded for autograd: gradients come from ``selective_scan_backward``, called
by hand.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._binding import (Library, On, check, check_float, check_whole, cuda_index, fit_ints, like,
                       out_dtype_of, raise_for, strides_of, workspace_of)
from .ttt_scan import IN_BF16, OUT_BF16

SSM_SOFTPLUS = 1 << 17
SSM_PAD_ZERO = 1 << 20
CHUNK = 16  # tokens between two snapshots of the state

_vp, _i, _u, _z = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_size_t
_lib = Library({
    "ttt_ssm_forward": ([_vp] * 10 + [_i] * 5 + [_u] + [_vp] * 5, _i),
    "ttt_ssm_backward_workspace_bytes": ([_i] * 5, _z),
    "ttt_ssm_backward": ([_vp] * 9 + [_i] * 5 + [_u] + [_vp] * 14 + [_z, _vp], _i),
    "ttt_ssm_step": ([_vp] * 10 + [_i] * 4 + [_u] + [_vp] * 3, _i),
})
_F32, _BF16 = torch.float32, torch.bfloat16
_ROWS, _TOKENS, _GROUPS = (0,), (0, 1), (0, 1, 2)  # dimensions whose strides count


def _mode(in_dtype, out_dtype, softplus, pad_zero) -> int:
    return ((IN_BF16 if in_dtype is _BF16 else 0) | (OUT_BF16 if out_dtype is _BF16 else 0) |
            (SSM_SOFTPLUS if softplus else 0) | (SSM_PAD_ZERO if pad_zero else 0))


def _check(u, delta, A, Bm, Cm, D, z, delta_bias, dims):
    """What every form takes, checked: device, G, N, Bm and Cm with their dimension of groups, and
    the addresses of u, delta, A, Bm, Cm, D, z, delta_bias."""
    dev, dtype, shape = cuda_index("u", u), u.dtype, u.shape
    if len(shape) != dims or A.dim() != 2:
        raise ValueError("u must be [B, T, D] (a step: [B, D]) and A [D, N]")
    N, C = A.shape[1], shape[-1]
    if Bm.dim() == dims:
        Bm, Cm = Bm.unsqueeze(-2), Cm.unsqueeze(-2)
    if Bm.dim() != dims + 1:
        raise ValueError("Bm must be [B, T, G, N] or [B, T, N] (a step: without T)")
    G = Bm.shape[-2]
    fit_ints("u, Bm", G, N, *shape)
    bc = shape[:-1] + (G, N)
    return dev, G, N, Bm, Cm, (
        check("u", u, shape, dtype, dev), check("delta", delta, shape, dtype, dev),
        check_whole("A", A, (C, N), _F32, dev), check("Bm", Bm, bc, dtype, dev),
        check("Cm", Cm, bc, dtype, dev), check_whole("D", D, (C,), _F32, dev),
        None if z is None else check("z", z, shape, dtype, dev),
        check_whole("delta_bias", delta_bias, (C,), _F32, dev))


def selective_scan(u, delta, A, Bm, Cm, D=None, z=None, delta_bias=None, *, softplus: bool = True,
                   h0=None, lengths=None, out_dtype: Optional[torch.dtype] = None,
                   want_chunks: bool = False, y: Optional[torch.Tensor] = None,
                   h_T: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None):
    """``(y, h_T) = selective_scan(u, delta, A, Bm, Cm, D, z, delta_bias)`` over a prompt.

    A: [D, N] fp32, N = 8, 16, 32 or 64; D, delta_bias: [D] fp32 or None (0); z: gate or None; h0: [B, D, N]
    fp32 state before the first token, or None (zeros); lengths: [B] int32 or None, the tokens of each
    row of a padded batch (those behind it are not read). y (``out_dtype``, default u's type) keeps
    its values behind a row's length; one made here is 0 there. h_T, the state after each row's last
    token, may be h0 itself. ``softplus=False`` takes delta + delta_bias as the step size.
    ``want_chunks`` also returns the states before every 16th token, [B, ceil(T/16), D, N], which
    ``selective_scan_backward`` starts from.
    """
    dev, G, N, Bm, Cm, ptrs = _check(u, delta, A, Bm, Cm, D, z, delta_bias, 3)
    B, T, C = u.shape
    h = check_whole("h0", h0, (B, C, N), _F32, dev)
    n = check_whole("lengths", lengths, (B,), torch.int32, dev)
    out_dtype = out_dtype_of(out_dtype, y, u.dtype)
    mode = _mode(u.dtype, out_dtype, softplus, y is None)
    chunks = None
    with On(dev, stream, (u, delta, A, Bm, Cm, D, z, delta_bias, h0, lengths, y, h_T)) as s:
        if y is None:
            y = like(delta, out_dtype)
        yp = check("y", y, u.shape, out_dtype, dev)
        if h_T is None:
            h_T = torch.empty((B, C, N), dtype=_F32, device=dev) if h0 is None else like(h0, _F32)
        hT = check_whole("h_T", h_T, (B, C, N), _F32, dev)
        if want_chunks:
            chunks = torch.empty((B, -(-T // CHUNK), C, N), dtype=_F32, device=dev)
        st = strides_of(14, (u, _TOKENS), (delta, _TOKENS), (u.shape if z is None else z, _TOKENS),
                        (Bm, _GROUPS), (Cm, _GROUPS), (y, _TOKENS))
        rc = _lib.ttt_ssm_forward(*ptrs, h, n, B, T, C, G, N, mode, st, yp, hT,
                                  None if chunks is None else chunks.data_ptr(), s)
    raise_for(rc, "ttt_ssm_forward")
    return (y, h_T, chunks) if want_chunks else (y, h_T)


def backward_workspace_bytes(B: int, T: int, D: int, G: int, N: int) -> int:
    """Bytes of device workspace ``ttt_ssm_backward`` needs for these sizes."""
    return int(_lib.ttt_ssm_backward_workspace_bytes(B, T, D, G, N))


def selective_scan_backward(u, delta, A, Bm, Cm, D, z, delta_bias, h_chunks, dy, dh_T=None, *,
                            softplus: bool = True, lengths=None,
                            workspace: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Gradients of ``<dy, y> + <dh_T, h_T>`` for a ``selective_scan`` with the same arguments.

    h_chunks: the snapshots of ``selective_scan(..., want_chunks=True)``; dy: as y (fp32 or bf16);
    dh_T: [B, D, N] fp32 or None (zero). Returns du, ddelta, dz (None without z), dBm, dCm (u's type; 0
    behind a row's length), dA, dD, ddelta_bias (None without the parameter) and dh0 (fp32).
    ``workspace`` (optional): at least ``backward_workspace_bytes`` bytes, not shared by calls that
    overlap.
    """
    bc_shape = Bm.shape
    dev, G, N, Bm, Cm, ptrs = _check(u, delta, A, Bm, Cm, D, z, delta_bias, 3)
    B, T, C = u.shape
    gp = check_float("dy", dy, u.shape, dev)
    ck = check_whole("h_chunks", h_chunks, (B, -(-T // CHUNK), C, N), _F32, dev)
    dh = check_whole("dh_T", dh_T, (B, C, N), _F32, dev)
    n = check_whole("lengths", lengths, (B,), torch.int32, dev)
    st = strides_of(14, (u, _TOKENS), (delta, _TOKENS), (u.shape if z is None else z, _TOKENS),
                    (Bm, _GROUPS), (Cm, _GROUPS), (dy, _TOKENS))
    with On(dev, stream, (u, delta, A, Bm, Cm, D, z, delta_bias, h_chunks, dy, dh_T, lengths,
                          workspace)) as s:
        workspace, wp, wn = workspace_of(workspace, backward_workspace_bytes(B, T, C, G, N), dev)
        act = dict(dtype=u.dtype, device=dev)
        out = dict(du=like(u, u.dtype), ddelta=like(u, u.dtype),
                   dz=None if z is None else like(u, u.dtype),
                   dBm=torch.empty(bc_shape, **act), dCm=torch.empty(bc_shape, **act),
                   dA=torch.empty_like(A), dD=None if D is None else torch.empty_like(D),
                   ddelta_bias=None if delta_bias is None else torch.empty_like(delta_bias),
                   dh0=torch.empty((B, C, N), dtype=_F32, device=dev))
        p = {k: None if v is None else v.data_ptr() for k, v in out.items()}
        rc = _lib.ttt_ssm_backward(
            *ptrs, n, B, T, C, G, N, _mode(u.dtype, dy.dtype, softplus, False), st, ck, gp, dh,
            p["du"], p["ddelta"], p["dA"], p["dBm"], p["dCm"], p["dD"], p["dz"], p["ddelta_bias"],
            p["dh0"], wp, wn, s)
    raise_for(rc, "ttt_ssm_backward")
    return out


def selective_step(u, delta, A, Bm, Cm, D, z, delta_bias, h, *, softplus: bool = True, active=None,
                   out_dtype: Optional[torch.dtype] = None, y: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None):
    """``y = selective_step(u, delta, A, Bm, Cm, D, z, delta_bias, h)``: one token of every row.

    u, delta, z: [B, D]; Bm, Cm: [B, G, N] or [B, N]; h: [B, D, N] fp32, updated IN PLACE; active: [B] uint8
    or None, 0 = the row's h and y are left as they were (a y made here is 0 there). D, z and
    delta_bias may be None. A chain of steps equals ``selective_scan``.
    """
    dev, G, N, Bm, Cm, ptrs = _check(u, delta, A, Bm, Cm, D, z, delta_bias, 2)
    B, C = u.shape
    if h is None:
        raise ValueError("h: expected the state")
    hp = check_whole("h", h, (B, C, N), _F32, dev)
    act = check_whole("active", active, (B,), torch.uint8, dev)
    out_dtype = out_dtype_of(out_dtype, y, u.dtype)
    mode = _mode(u.dtype, out_dtype, softplus, y is None)
    with On(dev, stream, (u, delta, A, Bm, Cm, D, z, delta_bias, h, active, y)) as s:
        if y is None:
            y = like(delta, out_dtype)
        yp = check("y", y, u.shape, out_dtype, dev)
        st = strides_of(8, (u, _ROWS), (delta, _ROWS), (u.shape if z is None else z, _ROWS),
                        (Bm, _TOKENS), (Cm, _TOKENS), (y, _ROWS))
        rc = _lib.ttt_ssm_step(*ptrs, hp, act, B, C, G, N, mode, st, yp, s)
    raise_for(rc, "ttt_ssm_step")
    return y
