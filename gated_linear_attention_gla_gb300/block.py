"""The parts of a recurrent block beside the mixers (argument marshalling only).

A gated linear recurrence with one state per channel, ``recur_*``; the norms, the
gate and the residual sum between two blocks, ``block_norm_*``; and the gated
feed-forward projections, ``glu_*`` (the down projection behind them is a plain
matrix product).  Each for prompts, for training (``*_bwd``: every gradient, from
the forward's inputs alone) and for single tokens (``recur_step`` on dense states
or a pool of pages; the others by their number of rows).  Formulas, layouts and
limits: ``include/gla.h``.

``x``, ``f``, ``i``, ``y`` and ``z`` may be column slices of one projection's
output (rows at one distance, 16-byte aligned); everything else is contiguous.
``stream`` as in ``ssm``.
"""
from __future__ import annotations

import torch

from ._binding import (GLA_FLAG_FP32_IO, GLA_FLAG_FP32_OUT, GLA_FLAG_FP32_RESIDUAL,
                       GLA_FLAG_LAYER_NORM, GLA_FLAG_UNIT_VARIANCE)
from ._marshal import (batch, check, counted, done, io_flags, launch_on, lib, output, page_tables, ptr,
                       rows, scratch, whole)

_F32 = torch.float32


def _recur_rows(x, f, decay, i, z):
    """Checks; the row arguments shared by the recurrence's entry points."""
    counted(x.shape[-1], "channels")
    check(x.is_cuda, "x must be a CUDA tensor")
    dev, ty, wide = x.device, x.dtype, x.shape
    pi, si = (None, 0) if i is None else rows(i, "i", wide, ty, dev)
    pz, sz = (None, 0) if z is None else rows(z, "z", wide, ty, dev)
    return (*rows(x, "x", wide, ty, dev), *rows(f, "f", wide, ty, dev), pi, si, pz, sz,
            whole(decay, "decay", (wide[-1],), _F32, dev))


def recur_fwd(x, f, decay=None, i=None, z=None, unit_variance: bool = True, init_state=None,
              cu_seqlens=None, out=None, final_state=None, output_final_state: bool = True,
              stream=None, out_dtype=None):
    """Gated linear recurrence of a prompt; returns ``(out, final_state)``.

    ``x``, ``f`` (forget gate), ``i`` (input gate, optional), ``z`` (output gate,
    optional): [B, T, D], or packed [1, R, D] / [R, D] with ``cu_seqlens`` (int32
    [B + 1] on the GPU), all before their activations.  ``decay`` (fp32 [D], <= 0):
    log a = decay sigmoid(f); None: a = sigmoid(f).  ``unit_variance``: the drive's
    factor is sqrt(1 - a^2), else 1 - a.  States are fp32 [B, D]; ``final_state``
    may be ``init_state``.  ``out`` has x's dtype, or fp32
    (``out_dtype=torch.float32``).
    """
    lead, B, T = batch(x, cu_seqlens, "x")
    D, dev, dt = x.shape[-1], x.device, x.dtype
    args = _recur_rows(x, f, decay, i, z)
    flags = io_flags(dt, out.dtype if out is not None else out_dtype or dt)
    flags |= GLA_FLAG_UNIT_VARIANCE if unit_variance else 0
    init = whole(init_state, "init_state", (B, D), _F32, dev)
    whole(final_state, "final_state", (B, D), _F32, dev)
    with launch_on(dev, stream) as s:
        out = output(out, x.shape, out_dtype or dt, dev)
        if final_state is None and output_final_state:
            final_state = torch.empty((B, D), dtype=_F32, device=dev)
        done(lib().gla_recur_fwd(*args, init, out.data_ptr(), ptr(final_state), ptr(cu_seqlens),
                                 B, T, D, s, flags), "gla_recur_fwd")
    return out, final_state


def recur_bwd(x, f, d_out, decay=None, i=None, z=None, unit_variance: bool = True,
              init_state=None, d_final_state=None, cu_seqlens=None, grad_dtype=None,
              need_d_init: bool = True, workspace=None, stream=None):
    """Gradient of ``recur_fwd``; returns ``(dx, df, d_decay, di, dz, d_init)``.

    ``d_out`` (x's shape and dtype, contiguous) and ``d_final_state`` (fp32 [B, D], or
    None for zero) are the gradients of the forward's outputs.  dx, df, di, dz
    come in x's dtype, or fp32 with ``grad_dtype=torch.float32``; d_decay and d_init
    are fp32; gradients of what was not given are None.
    """
    lead, B, T = batch(x, cu_seqlens, "x")
    D, dev = x.shape[-1], x.device
    args = _recur_rows(x, f, decay, i, z)
    grad_dtype = grad_dtype or x.dtype
    flags = io_flags(x.dtype, grad_dtype) | (GLA_FLAG_UNIT_VARIANCE if unit_variance else 0)
    init = whole(init_state, "init_state", (B, D), _F32, dev)
    dy = whole(d_out, "d_out", x.shape, x.dtype, dev)
    df_ = whole(d_final_state, "d_final_state", (B, D), _F32, dev)
    with launch_on(dev, stream) as s:
        size = lib().gla_recur_bwd_workspace_size(B, T, D, cu_seqlens is not None)
        workspace = scratch(size, workspace, dev)
        new = lambda shape, dtype=_F32: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        dx, df = new(x.shape, grad_dtype), new(x.shape, grad_dtype)
        di = new(x.shape, grad_dtype) if i is not None else None
        dz = new(x.shape, grad_dtype) if z is not None else None
        dd = new(D) if decay is not None else None
        d0 = new((B, D)) if need_d_init else None
        done(lib().gla_recur_bwd(*args, init, dy, df_, dx.data_ptr(), df.data_ptr(), ptr(di),
                                 ptr(dz), ptr(dd), ptr(d0), ptr(cu_seqlens), B, T, D,
                                 ptr(workspace), size, s, flags), "gla_recur_bwd")
    return dx, df, dd, di, dz, d0


def recur_step(x, f, state, decay=None, i=None, z=None, unit_variance: bool = True, slots=None,
               out_slots=None, out=None, stream=None, out_dtype=None):
    """One token for N sequences: ``x``, ``f``, ``i``, ``z`` [N, D]; returns ``out`` [N, D].
    ``state`` (fp32 [N, D]) is updated in place; with ``slots`` and ``out_slots`` it is a
    pool [num_slots, D], as for ``conv_step``."""
    check(x.dim() == 2, "x is [N, D]")
    (N, D), dev, dt = x.shape, x.device, x.dtype
    n = counted(N, "rows")
    args = _recur_rows(x, f, decay, i, z)
    if slots is not None:
        n = counted(state.shape[0], "pages") if state.dim() else 0
    ps = whole(state, "state", (n, D), _F32, dev)
    pi, po = page_tables(N, dev, slots, out_slots)
    flags = io_flags(dt, out.dtype if out is not None else out_dtype or dt)
    flags |= GLA_FLAG_UNIT_VARIANCE if unit_variance else 0
    with launch_on(dev, stream) as s:
        out = output(out, (N, D), out_dtype or dt, dev)
        done(lib().gla_recur_step(*args, ps, 0 if slots is None else n, pi, po, out.data_ptr(),
                                  N, D, s, flags), "gla_recur_step")
    return out


def _norm_rows(res, y, z, post_weight, post_bias, scale, weight, bias, kind, dtype):
    """Checks; (D, rows, flags, the leading row arguments, the parameters' addresses)."""
    check(res.dim() in (2, 3), "res is [R, D] or [B, T, D]")
    R, D = counted(res.shape[:-1].numel(), "rows"), counted(res.shape[-1], "channels")
    check(res.is_cuda, "res must be a CUDA tensor")
    check(kind in ("rms", "layer"), 'kind is "rms" or "layer"')
    dev, wide = res.device, res.shape
    if dtype is torch.float32:
        flags = GLA_FLAG_FP32_IO
    else:
        check(dtype is torch.bfloat16, "rows must be bf16 or fp32")
        flags = 0 if res.dtype is dtype else GLA_FLAG_FP32_RESIDUAL
    flags |= GLA_FLAG_LAYER_NORM if kind == "layer" else 0
    check(res.dtype in (dtype, _F32), "res has y's dtype, or fp32")
    check(y is not None or (z is None and post_weight is None and post_bias is None and
                            scale is None), "z, post_weight, post_bias and scale need y")
    py, sy = (None, 0) if y is None else rows(y, "y", wide, dtype, dev)
    pz, sz = (None, 0) if z is None else rows(z, "z", wide, dtype, dev)
    par = [whole(t, name, (D,), _F32, dev) for name, t in (
        ("post_weight", post_weight), ("post_bias", post_bias), ("scale", scale),
        ("weight", weight), ("bias", bias))]
    return D, R, flags, (whole(res, "res", wide, res.dtype, dev), py, sy, pz, sz), par


def block_norm_fwd(res, y=None, z=None, post_weight=None, post_bias=None, scale=None, weight=None,
                   bias=None, kind: str = "rms", eps: float = 1e-6, res_out=None, out=None,
                   stream=None, out_dtype=None):
    """Between two blocks; returns ``(res_out, out)``:

        p = norm(y) post_weight + post_bias;  s = res + scale p silu(z);  out = norm(s) weight + bias

    ``y``, ``z`` [.., D] (bf16 or fp32), ``res`` of that dtype or fp32; the parameters fp32
    [D], each left out where None; ``kind`` "rms" or "layer".  Without ``y`` it is
    the norm of ``res`` alone and ``res_out`` is None; without ``weight`` it ends at the
    sum and ``out`` is None.  ``res_out`` may be ``res`` (in place).  ``out`` has y's
    dtype; ``out_dtype=torch.float32`` or bf16 overrides it (and names the rows' dtype
    where there is no y).
    """
    if out is not None:
        out_dtype = out.dtype
    dtype = y.dtype if y is not None else out_dtype or res.dtype
    if y is None and res.dtype is torch.bfloat16:
        dtype = torch.bfloat16
    D, R, flags, lead, par = _norm_rows(res, y, z, post_weight, post_bias, scale, weight, bias,
                                        kind, dtype)
    dev = res.device
    out_dtype = out_dtype or dtype
    check(out_dtype is dtype or (dtype is torch.bfloat16 and out_dtype is _F32),
          "out has y's dtype, or fp32")
    if out_dtype is not dtype:
        flags |= GLA_FLAG_FP32_OUT
    check(weight is not None or (bias is None and out is None), "bias and out need weight")
    check(y is not None or res_out is None, "res_out needs y")
    if res_out is not None:
        whole(res_out, "res_out", res.shape, res.dtype, dev)
    with launch_on(dev, stream) as s:
        if res_out is None and y is not None:
            res_out = torch.empty_like(res, memory_format=torch.contiguous_format)
        if weight is not None:
            out = output(out, res.shape, out_dtype, dev)
        done(lib().gla_block_norm_fwd(*lead, *par, eps, ptr(res_out), ptr(out), R, D, s, flags),
             "gla_block_norm_fwd")
    return res_out, out


def block_norm_bwd(res, d_out=None, d_res_out=None, y=None, z=None, post_weight=None,
                   post_bias=None, scale=None, weight=None, bias=None, kind: str = "rms",
                   eps: float = 1e-6, grad_dtype=None, workspace=None, stream=None):
    """Gradient of ``block_norm_fwd``; returns ``(d_res, dy, dz, d_post_weight, d_post_bias,
    d_scale, d_weight, d_bias)``.

    ``d_out`` (the rows' dtype) and ``d_res_out`` (res's dtype) are the gradients of the
    forward's outputs, contiguous, None for zero.  d_res comes in res's dtype, dy
    and dz in y's, all fp32 with ``grad_dtype=torch.float32``; the parameters' gradients
    are fp32; gradients of what was not given are None, and without ``d_out`` those of
    ``weight`` and ``bias`` (which are zero) too.
    """
    dtype = y.dtype if y is not None else d_out.dtype if d_out is not None else res.dtype
    check(d_out is None or weight is not None, "d_out needs weight")
    if d_out is None:
        weight = bias = None
    D, R, flags, lead, par = _norm_rows(res, y, z, post_weight, post_bias, scale, weight, bias,
                                        kind, dtype)
    dev = res.device
    grad_dtype = grad_dtype or dtype
    check(grad_dtype is dtype or (dtype is torch.bfloat16 and grad_dtype is _F32),
          "gradients come in the rows' dtype, or fp32")
    if grad_dtype is not dtype:
        flags |= GLA_FLAG_FP32_OUT
    du = whole(d_out, "d_out", res.shape, dtype, dev)
    ds = whole(d_res_out, "d_res_out", res.shape, res.dtype, dev)
    with launch_on(dev, stream) as s:
        size = lib().gla_block_norm_bwd_workspace_size(R, D)
        workspace = scratch(size, workspace, dev)
        new = lambda dt: torch.empty(res.shape, dtype=dt, device=dev)  # noqa: E731
        d_res = new(_F32 if grad_dtype is _F32 else res.dtype)
        dy = new(grad_dtype) if y is not None else None
        dz = new(grad_dtype) if z is not None else None
        vec = [None if t is None else torch.empty(D, dtype=_F32, device=dev)
               for t in (post_weight, post_bias, scale, weight, bias)]
        done(lib().gla_block_norm_bwd(*lead, *par[:4], eps, du, ds, d_res.data_ptr(), ptr(dy),
                                      ptr(dz), *map(ptr, vec), R, D, ptr(workspace), size, s,
                                      flags), "gla_block_norm_bwd")
    return (d_res, dy, dz, *vec)


def _glu_rows(x, w_gate, w_up):
    """Checks; (R, D, F, the leading arguments)."""
    check(x.dim() in (2, 3) and w_gate.dim() == 2, "x is [R, D] or [B, T, D], weights are [F, D]")
    R, D = counted(x.shape[:-1].numel(), "rows"), counted(x.shape[-1], "channels")
    F = counted(w_gate.shape[0], "features")
    check(x.is_cuda, "x must be a CUDA tensor")
    check(x.dtype is torch.bfloat16, "the projections are bf16")
    dev = x.device
    return R, D, F, (
        *rows(x, "x", x.shape, x.dtype, dev), whole(w_gate, "w_gate", (F, D), x.dtype, dev),
        whole(w_up, "w_up", (F, D), x.dtype, dev))


def glu_fwd(x, w_gate, w_up, out=None, stream=None, out_dtype=None):
    """silu(x w_gate^T) * (x w_up^T): ``x`` [.., D], ``w_gate``, ``w_up`` [F, D] (bf16);
    returns ``out`` [.., F] in bf16, or fp32 (``out_dtype=torch.float32``)."""
    R, D, F, args = _glu_rows(x, w_gate, w_up)
    out_dtype = out.dtype if out is not None else out_dtype or x.dtype
    flags = io_flags(x.dtype, out_dtype)
    with launch_on(x.device, stream) as s:
        out = output(out, (*x.shape[:-1], F), out_dtype, x.device)
        done(lib().gla_glu_fwd(*args, out.data_ptr(), R, D, F, s, flags), "gla_glu_fwd")
    return out


def glu_bwd(x, w_gate, w_up, d_out, grad_dtype=None, workspace=None, stream=None):
    """Gradient of ``glu_fwd``; returns ``(dx, dw_gate, dw_up)``.  ``d_out`` [.., F] in bf16,
    contiguous; the gradients come in bf16, or fp32 with ``grad_dtype=torch.float32``.  At most
    2^26 rows."""
    R, D, F, args = _glu_rows(x, w_gate, w_up)
    dev = x.device
    grad_dtype = grad_dtype or x.dtype
    flags = io_flags(x.dtype, grad_dtype)
    dh = whole(d_out, "d_out", (*x.shape[:-1], F), x.dtype, dev)
    with launch_on(dev, stream) as s:
        size = lib().gla_glu_bwd_workspace_size(R, D, F)
        workspace = scratch(size, workspace, dev)
        dx = torch.empty(x.shape, dtype=grad_dtype, device=dev)
        dg, du = (torch.empty((F, D), dtype=grad_dtype, device=dev) for _ in range(2))
        done(lib().gla_glu_bwd(*args, dh, dx.data_ptr(), dg.data_ptr(), du.data_ptr(), R, D, F,
                               ptr(workspace), size, s, flags), "gla_glu_bwd")
    return dx, dg, du
