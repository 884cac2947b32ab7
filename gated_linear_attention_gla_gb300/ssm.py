"""The selective-scan layer's parts that carry state (argument marshalling only).

A short causal convolution per channel, ``conv_*``, and a state space scan whose
decay and drive depend on the token, ``scan_*``, each for prompts (dense, or
packed with ``cu_seqlens``), for training (``*_bwd``: every gradient, from the
forward's inputs alone) and for single tokens (``*_step``, on dense states or on
a pool of pages).  Formulas, layouts and limits: ``include/gla.h``.

``x``, ``u``, ``dt``, ``z``, ``b`` and ``c`` may be column slices of one
projection's output (rows at one distance, 16-byte aligned except for b and c);
everything else is contiguous.  Parameters and their gradients are fp32, the
convolution's states have x's dtype, the scan's are fp32.  Call arguments given
as ``stream`` run the call (and what it allocates) on that stream.
"""
from __future__ import annotations

from typing import Optional

import torch

from ._binding import GLA_FLAG_SILU, GLA_FLAG_SOFTPLUS
from ._marshal import (batch, check, counted, done, io_flags, launch_on, lib, output, page_tables,
                       ptr, rows, scratch, whole)

_F32 = torch.float32


def _silu_flag(activation) -> int:
    check(activation in (None, "silu"), 'activation is None or "silu"')
    return GLA_FLAG_SILU if activation else 0


def _state(state, n, a, b, dtype, device, slots):
    """The address of a state, dense or a pool, and the pool's pages."""
    shape = state.shape
    if len(shape) != 3 or shape[1] != a or shape[2] != b or state.dtype is not dtype or \
            state.device != device or not state.is_contiguous() or \
            (slots is None and shape[0] != n):
        raise ValueError(f"state must be contiguous {dtype} "
                         f"[{n if slots is None else 'num_slots'}, {a}, {b}] on {device}")
    return state.data_ptr(), 0 if slots is None else counted(shape[0], "pages")


def _filter(x, weight, bias):
    """(D, W, the filter's and the bias's addresses)."""
    D, dev = counted(x.shape[-1], "channels"), x.device
    check(x.is_cuda, "x must be a CUDA tensor")
    check(weight.dim() == 2, "weight is [D, W]")
    W = weight.shape[1]
    return (D, W, whole(weight, "weight", (D, W), _F32, dev),
            whole(bias, "bias", (D,), _F32, dev))


def conv_fwd(x, weight, bias=None, init_state=None, cu_seqlens=None,
             activation: Optional[str] = None, out=None, final_state=None,
             output_final_state: bool = True, stream=None, out_dtype=None):
    """Causal convolution of a prompt; returns ``(out, final_state)``.

    ``x`` [B, T, D], or packed [1, R, D] / [R, D] with ``cu_seqlens`` (int32
    [B + 1] on the GPU); ``weight`` [D, W] (W = 2, 3, 4; column W - 1 meets the
    token itself) and ``bias`` [D], fp32; ``activation`` None or "silu";
    ``init_state`` and ``final_state`` [B, W - 1, D] in x's dtype, the last W - 1
    inputs (oldest first).  ``out`` has x's dtype, or fp32
    (``out_dtype=torch.float32``); ``final_state`` may be ``init_state``.
    """
    lead, B, T = batch(x, cu_seqlens, "x")
    D, W, w, b = _filter(x, weight, bias)
    dev, dt, st = x.device, x.dtype, (B, W - 1, D)
    px, stride = rows(x, "x", x.shape, dt, dev)
    flags = io_flags(dt, out.dtype if out is not None else out_dtype or dt)
    flags |= _silu_flag(activation)
    init = whole(init_state, "init_state", st, dt, dev)
    whole(final_state, "final_state", st, dt, dev)
    with launch_on(dev, stream) as s:
        out = output(out, x.shape, out_dtype or dt, dev)
        if final_state is None and output_final_state:
            final_state = torch.empty(st, dtype=dt, device=dev)
        done(lib().gla_conv_fwd(px, stride, w, b, init, out.data_ptr(), ptr(final_state),
                                ptr(cu_seqlens), B, T, D, W, s, flags), "gla_conv_fwd")
    return out, final_state


def conv_bwd(x, weight, d_out, bias=None, init_state=None, d_final_state=None, cu_seqlens=None,
             activation: Optional[str] = None, grad_dtype=None, need_d_init: bool = True,
             workspace=None, stream=None):
    """Gradient of ``conv_fwd``; returns ``(dx, d_weight, d_bias, d_init)``.

    ``d_out`` (x's shape and dtype, contiguous) and ``d_final_state`` (fp32
    [B, W - 1, D], or None for zero) are the gradients of the forward's outputs.
    ``dx`` has x's dtype, or fp32 with ``grad_dtype=torch.float32``; ``d_bias`` is
    None without a bias; ``d_init`` is fp32 (None when not requested).
    """
    lead, B, T = batch(x, cu_seqlens, "x")
    D, W, w, b = _filter(x, weight, bias)
    dev, dt, st = x.device, x.dtype, (B, W - 1, D)
    px, stride = rows(x, "x", x.shape, dt, dev)
    grad_dtype = grad_dtype or dt
    flags = io_flags(dt, grad_dtype) | _silu_flag(activation)
    init = whole(init_state, "init_state", st, dt, dev)
    dy = whole(d_out, "d_out", x.shape, dt, dev)
    df = whole(d_final_state, "d_final_state", st, _F32, dev)
    with launch_on(dev, stream) as s:
        size = lib().gla_conv_bwd_workspace_size(B, T, D, W, cu_seqlens is not None)
        workspace = scratch(size, workspace, dev)
        dx = torch.empty(x.shape, dtype=grad_dtype, device=dev)
        dw = torch.empty((D, W), dtype=_F32, device=dev)
        db = torch.empty(D, dtype=_F32, device=dev) if bias is not None else None
        di = torch.empty(st, dtype=_F32, device=dev) if need_d_init else None
        done(lib().gla_conv_bwd(px, stride, w, b, init, dy, df, dx.data_ptr(), dw.data_ptr(),
                                ptr(db), ptr(di), ptr(cu_seqlens), B, T, D, W, ptr(workspace),
                                size, s, flags), "gla_conv_bwd")
    return dx, dw, db, di


def conv_step(x, weight, state, bias=None, activation: Optional[str] = None, slots=None,
              out_slots=None, out=None, stream=None, out_dtype=None):
    """One token for N sequences: ``x`` [N, D]; returns ``out`` [N, D].

    ``state`` [N, W - 1, D] in x's dtype is shifted by x in place.  With
    ``slots`` (int32 [N] on the GPU) it is a pool [num_slots, W - 1, D]: row n
    reads page ``slots[n]`` and writes it, or page ``out_slots[n]`` where that is
    given (the page read stays as it was).  -1 in either marks a row that does
    nothing.
    """
    check(x.dim() == 2, "x is [N, D]")
    N, dev, dt = counted(x.shape[0], "rows"), x.device, x.dtype
    D, W, w, b = _filter(x, weight, bias)
    px, stride = rows(x, "x", x.shape, dt, dev)
    ps, pages = _state(state, N, W - 1, D, dt, dev, slots)
    pi, po = page_tables(N, dev, slots, out_slots)
    flags = io_flags(dt, out.dtype if out is not None else out_dtype or dt)
    flags |= _silu_flag(activation)
    with launch_on(dev, stream) as s:
        out = output(out, (N, D), out_dtype or dt, dev)
        done(lib().gla_conv_step(px, stride, w, b, ps, pages, pi, po, out.data_ptr(), N, D, W, s,
                                 flags), "gla_conv_step")
    return out


def _scan_common(u, dt, a, b, c, skip, z, dt_bias, lead):
    """Checks; returns (D, N, the row arguments shared by the scan's entry points)."""
    dev, ty, wide = u.device, u.dtype, u.shape
    D, N = counted(wide[-1], "channels"), a.shape[-1]
    check(u.is_cuda, "u must be a CUDA tensor")
    narrow = (*lead, N)
    pz, sz = (None, 0) if z is None else rows(z, "z", wide, ty, dev)
    return D, N, (*rows(u, "u", wide, ty, dev), *rows(dt, "dt", wide, ty, dev),
                  whole(a, "a", (D, N), _F32, dev), *rows(b, "b", narrow, ty, dev),
                  *rows(c, "c", narrow, ty, dev), whole(skip, "skip", (D,), _F32, dev), pz, sz,
                  whole(dt_bias, "dt_bias", (D,), _F32, dev))


def scan_fwd(u, dt, a, b, c, skip=None, z=None, dt_bias=None, softplus: bool = True,
             init_state=None, cu_seqlens=None, out=None, final_state=None,
             output_final_state: bool = True, workspace=None, stream=None, out_dtype=None):
    """Selective scan of a prompt; returns ``(out, final_state)``.

    ``u``, ``dt``, ``z`` [B, T, D] (packed: [1, R, D] or [R, D] with
    ``cu_seqlens``), ``b``, ``c`` [.., N] with N = 8, 16, 32 or 64, all in u's
    dtype; ``a`` [D, N], ``skip`` [D], ``dt_bias`` [D] fp32.  ``softplus``: the
    step size is softplus(dt + dt_bias), else their sum.  States are fp32
    [B, D, N]; ``final_state`` may be ``init_state``.  ``out`` has u's dtype, or
    fp32 (``out_dtype=torch.float32``).  ``workspace``: a uint8 tensor of
    gla_scan_fwd_workspace_size bytes, or None for a fresh one.
    """
    lead, B, T = batch(u, cu_seqlens, "u")
    D, N, args = _scan_common(u, dt, a, b, c, skip, z, dt_bias, lead)
    dev = u.device
    flags = io_flags(u.dtype, out.dtype if out is not None else out_dtype or u.dtype)
    flags |= GLA_FLAG_SOFTPLUS if softplus else 0
    init = whole(init_state, "init_state", (B, D, N), _F32, dev)
    whole(final_state, "final_state", (B, D, N), _F32, dev)
    with launch_on(dev, stream) as s:
        size = lib().gla_scan_fwd_workspace_size(B, T, D, N, cu_seqlens is not None)
        workspace = scratch(size, workspace, dev)
        out = output(out, u.shape, out_dtype or u.dtype, dev)
        if final_state is None and output_final_state:
            final_state = torch.empty((B, D, N), dtype=_F32, device=dev)
        done(lib().gla_scan_fwd(*args, init, out.data_ptr(), ptr(final_state), ptr(cu_seqlens),
                                B, T, D, N, ptr(workspace), size, s, flags), "gla_scan_fwd")
    return out, final_state


def scan_bwd(u, dt, a, b, c, d_out, skip=None, z=None, dt_bias=None, softplus: bool = True,
             init_state=None, d_final_state=None, cu_seqlens=None, grad_dtype=None,
             need_d_init: bool = True, workspace=None, stream=None):
    """Gradient of ``scan_fwd``; returns ``(du, ddt, da, db, dc, dskip, dz, ddt_bias, d_init)``.

    ``d_out`` (u's shape and dtype, contiguous) and ``d_final_state`` (fp32 state,
    or None for zero) are the gradients of the forward's outputs.  du, ddt, db,
    dc, dz come in u's dtype, or fp32 with ``grad_dtype=torch.float32``; da, dskip,
    ddt_bias and d_init are fp32; gradients of what was not given are None.
    """
    lead, B, T = batch(u, cu_seqlens, "u")
    D, N, args = _scan_common(u, dt, a, b, c, skip, z, dt_bias, lead)
    dev = u.device
    grad_dtype = grad_dtype or u.dtype
    flags = io_flags(u.dtype, grad_dtype) | (GLA_FLAG_SOFTPLUS if softplus else 0)
    init = whole(init_state, "init_state", (B, D, N), _F32, dev)
    dy = whole(d_out, "d_out", u.shape, u.dtype, dev)
    df = whole(d_final_state, "d_final_state", (B, D, N), _F32, dev)
    with launch_on(dev, stream) as s:
        size = lib().gla_scan_bwd_workspace_size(B, T, D, N, cu_seqlens is not None)
        workspace = scratch(size, workspace, dev)
        new = lambda shape, dtype=_F32: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        du, ddt = new(u.shape, grad_dtype), new(u.shape, grad_dtype)
        db, dc = new(b.shape, grad_dtype), new(c.shape, grad_dtype)
        dz = new(u.shape, grad_dtype) if z is not None else None
        da = new((D, N))
        dskip = new(D) if skip is not None else None
        dbias = new(D) if dt_bias is not None else None
        di = new((B, D, N)) if need_d_init else None
        done(lib().gla_scan_bwd(*args, init, dy, df, du.data_ptr(), ddt.data_ptr(),
                                da.data_ptr(), db.data_ptr(), dc.data_ptr(), ptr(dskip), ptr(dz),
                                ptr(dbias), ptr(di), ptr(cu_seqlens), B, T, D, N, ptr(workspace),
                                size, s, flags), "gla_scan_bwd")
    return du, ddt, da, db, dc, dskip, dz, dbias, di


def scan_step(u, dt, a, b, c, state, skip=None, z=None, dt_bias=None, softplus: bool = True,
              slots=None, out_slots=None, out=None, stream=None, out_dtype=None):
    """One token for R sequences: ``u``, ``dt``, ``z`` [R, D], ``b``, ``c`` [R, N]; returns
    ``out`` [R, D].  ``state`` (fp32 [R, D, N]) is updated in place; with ``slots``
    and ``out_slots`` it is a pool [num_slots, D, N], as for ``conv_step``."""
    check(u.dim() == 2, "u is [R, D]")
    R = counted(u.shape[0], "rows")
    D, N, args = _scan_common(u, dt, a, b, c, skip, z, dt_bias, (R,))
    dev = u.device
    ps, pages = _state(state, R, D, N, _F32, dev, slots)
    pi, po = page_tables(R, dev, slots, out_slots)
    flags = io_flags(u.dtype, out.dtype if out is not None else out_dtype or u.dtype)
    flags |= GLA_FLAG_SOFTPLUS if softplus else 0
    with launch_on(dev, stream) as s:
        out = output(out, (R, D), out_dtype or u.dtype, dev)
        done(lib().gla_scan_step(*args, ps, pages, pi, po, out.data_ptr(), R, D, N, s, flags),
             "gla_scan_step")
    return out
