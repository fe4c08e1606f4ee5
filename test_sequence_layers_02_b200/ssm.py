"""Selective state space scan (``include/ttt_ssm.h``), a sibling of the TTT scan whose state is N numbers for
each channel:

    dt_t = softplus(delta_t + delta_bias)
    h_t  = exp(dt_t A) h_{t-1} + dt_t u_t Bm_t,   y_t = (Cm_t . h_t + D u_t) SiLU(z_t)

for prompts (``selective_scan``), training (``selective_scan_backward``) and single tokens
(``selective_step``). u, delta, z, y are [B, T, D], Bm and Cm [B, T, G, N] (or [B, T, N] for one
group), fp32 or bf16, with contiguous rows and any strides between batch rows, tokens and groups;
parameters and states are fp32. CUDA tensors only; see ``_binding`` for streams. There is no CPU
fallback.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._binding import (Library, On, check, check_device, check_dtype, check_whole, out_dtype_of,
                       raise_for, strides_of)
from .ttt_scan import IN_BF16, OUT_BF16

SSM_SOFTPLUS = 1 << 17
CHUNK = 16  # tokens between two snapshots of the state

_vp, _i, _u, _z = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_size_t
_lib = Library({
    "ttt_ssm_forward": ([_vp] * 10 + [_i] * 5 + [_u] + [_vp] * 5, _i),
    "ttt_ssm_backward_workspace_bytes": ([_i] * 5, _z),
    "ttt_ssm_backward": ([_vp] * 9 + [_i] * 5 + [_u] + [_vp] * 14 + [_z, _vp], _i),
    "ttt_ssm_step": ([_vp] * 10 + [_i] * 4 + [_u] + [_vp] * 3, _i),
})


def _mode(in_dtype, out_dtype, softplus) -> int:
    return ((IN_BF16 if in_dtype == torch.bfloat16 else 0) |
            (OUT_BF16 if out_dtype == torch.bfloat16 else 0) | (SSM_SOFTPLUS if softplus else 0))


def _check(u, delta, A, Bm, Cm, D, z, delta_bias):
    """Shapes and types of what every form takes. Bm and Cm come back with their group dimension."""
    dev, dtype = check_device("u", u), check_dtype("u", u)
    if A.dim() != 2:
        raise ValueError("A must be [D, N]")
    N = A.shape[1]
    check("u", u, u.shape, dtype, dev)
    check("delta", delta, u.shape, dtype, dev)
    if z is not None:
        check("z", z, u.shape, dtype, dev)
    if Bm.dim() == u.dim():
        Bm, Cm = Bm.unsqueeze(-2), Cm.unsqueeze(-2)
    if Bm.dim() != u.dim() + 1:
        raise ValueError("Bm must be [B, T, G, N] or [B, T, N] (a step: without T)")
    G = Bm.shape[-2]
    shape = u.shape[:-1] + (G, N)
    check("Bm", Bm, shape, dtype, dev)
    check("Cm", Cm, shape, dtype, dev)
    ch = (u.shape[-1],)
    pars = (check_whole("A", A, ch + (N,), torch.float32, dev),
            check_whole("D", D, ch, torch.float32, dev),
            check_whole("delta_bias", delta_bias, ch, torch.float32, dev))
    return dev, dtype, G, N, Bm, Cm, pars


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
    if u.dim() != 3:
        raise ValueError("u must be [B, T, D]")
    dev, dtype, G, N, Bm, Cm, (a, d, bias) = _check(u, delta, A, Bm, Cm, D, z, delta_bias)
    B, T, C = u.shape
    h = check_whole("h0", h0, (B, C, N), torch.float32, dev)
    n = check_whole("lengths", lengths, (B,), torch.int32, dev)
    out_dtype = out_dtype_of(out_dtype if y is None else y.dtype, dtype)
    chunks = None
    with On(dev, stream, (u, delta, A, Bm, Cm, D, z, delta_bias, h0, lengths, y, h_T)) as s:
        if y is None:
            make = torch.empty if lengths is None else torch.zeros
            y = make(u.shape, dtype=out_dtype, device=dev)
        else:
            check("y", y, u.shape, out_dtype, dev)
        if h_T is None:
            h_T = torch.empty((B, C, N), dtype=torch.float32, device=dev)
        hT = check_whole("h_T", h_T, (B, C, N), torch.float32, dev)
        if want_chunks:
            chunks = torch.empty((B, -(-T // CHUNK), C, N), dtype=torch.float32, device=dev)
        st = strides_of((u, (0, 1)), (delta, (0, 1)), (u.shape if z is None else z, (0, 1)),
                        (Bm, (0, 1, 2)), (Cm, (0, 1, 2)), (y, (0, 1)))
        rc = _lib().ttt_ssm_forward(
            u.data_ptr(), delta.data_ptr(), a, Bm.data_ptr(), Cm.data_ptr(), d,
            None if z is None else z.data_ptr(), bias, h, n, B, T, C, G, N,
            _mode(dtype, out_dtype, softplus), st, y.data_ptr(), hT,
            None if chunks is None else chunks.data_ptr(), s)
    raise_for(rc, "ttt_ssm_forward")
    return (y, h_T, chunks) if want_chunks else (y, h_T)


def backward_workspace_bytes(B: int, T: int, D: int, G: int, N: int) -> int:
    """Bytes of device workspace ``ttt_ssm_backward`` needs for these sizes."""
    return int(_lib().ttt_ssm_backward_workspace_bytes(B, T, D, G, N))


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
    if u.dim() != 3:
        raise ValueError("u must be [B, T, D]")
    bc_shape = Bm.shape
    dev, dtype, G, N, Bm, Cm, (a, d, bias) = _check(u, delta, A, Bm, Cm, D, z, delta_bias)
    B, T, C = u.shape
    check("dy", dy, u.shape, check_dtype("dy", dy), dev)
    ck = check_whole("h_chunks", h_chunks, (B, -(-T // CHUNK), C, N), torch.float32, dev)
    dh = check_whole("dh_T", dh_T, (B, C, N), torch.float32, dev)
    n = check_whole("lengths", lengths, (B,), torch.int32, dev)
    st = strides_of((u, (0, 1)), (delta, (0, 1)), (u.shape if z is None else z, (0, 1)),
                    (Bm, (0, 1, 2)), (Cm, (0, 1, 2)), (dy, (0, 1)))
    with On(dev, stream, (u, delta, A, Bm, Cm, D, z, delta_bias, h_chunks, dy, dh_T, lengths,
                          workspace)) as s:
        need = backward_workspace_bytes(B, T, C, G, N)
        if workspace is None:
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        check_whole("workspace", workspace, workspace.shape, workspace.dtype, dev)
        act = dict(dtype=dtype, device=dev)
        out = dict(du=torch.empty(u.shape, **act), ddelta=torch.empty(u.shape, **act),
                   dz=None if z is None else torch.empty(u.shape, **act),
                   dBm=torch.empty(bc_shape, **act), dCm=torch.empty(bc_shape, **act),
                   dA=torch.empty_like(A), dD=None if D is None else torch.empty_like(D),
                   ddelta_bias=None if delta_bias is None else torch.empty_like(delta_bias),
                   dh0=torch.empty((B, C, N), dtype=torch.float32, device=dev))
        p = {k: None if v is None else v.data_ptr() for k, v in out.items()}
        rc = _lib().ttt_ssm_backward(
            u.data_ptr(), delta.data_ptr(), a, Bm.data_ptr(), Cm.data_ptr(), d,
            None if z is None else z.data_ptr(), bias, n, B, T, C, G, N,
            _mode(dtype, dy.dtype, softplus), st, ck, dy.data_ptr(), dh, p["du"], p["ddelta"],
            p["dA"], p["dBm"], p["dCm"], p["dD"], p["dz"], p["ddelta_bias"], p["dh0"],
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), s)
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
    if u.dim() != 2:
        raise ValueError("u must be [B, D]")
    dev, dtype, G, N, Bm, Cm, (a, d, bias) = _check(u, delta, A, Bm, Cm, D, z, delta_bias)
    B, C = u.shape
    if h is None:
        raise ValueError("h: expected the state")
    hp = check_whole("h", h, (B, C, N), torch.float32, dev)
    act = check_whole("active", active, (B,), torch.uint8, dev)
    out_dtype = out_dtype_of(out_dtype if y is None else y.dtype, dtype)
    with On(dev, stream, (u, delta, A, Bm, Cm, D, z, delta_bias, h, active, y)) as s:
        if y is None:
            make = torch.empty if active is None else torch.zeros
            y = make(u.shape, dtype=out_dtype, device=dev)
        else:
            check("y", y, u.shape, out_dtype, dev)
        st = strides_of((u, (0,)), (delta, (0,)), (u.shape if z is None else z, (0,)),
                        (Bm, (0, 1)), (Cm, (0, 1)), (y, (0,)))
        rc = _lib().ttt_ssm_step(
            u.data_ptr(), delta.data_ptr(), a, Bm.data_ptr(), Cm.data_ptr(), d,
            None if z is None else z.data_ptr(), bias, hp, act, B, C, G, N,
            _mode(dtype, out_dtype, softplus), st, y.data_ptr(), s)
    raise_for(rc, "ttt_ssm_step")
    return y
