"""Argument marshalling shared by ``ssm`` and ``pages``: checks, row strides,
the device and stream a call runs on."""
from __future__ import annotations

import torch

from . import _binding
from ._binding import GLA_FLAG_FP32_IO, GLA_FLAG_FP32_OUT, GlaError


def check(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


def ptr(t) -> int:
    return None if t is None else t.data_ptr()


class launch_on:
    """The stream a call launches on, as an int: the tensors' device made current, and
    ``stream`` (default: that device's current stream) too, so that what the call
    allocates belongs to the stream it is used on."""

    __slots__ = ("device", "stream", "guards")

    def __init__(self, device, stream):
        self.device, self.stream, self.guards = device, stream, ()

    def __enter__(self) -> int:
        if self.device.index != torch.cuda.current_device():
            self.guards = (torch.cuda.device(self.device),)
            self.guards[0].__enter__()
        if self.stream is None:
            return torch.cuda.current_stream().cuda_stream
        s = self.stream
        if not isinstance(s, torch.cuda.Stream):
            s = torch.cuda.ExternalStream(int(s), device=self.device) if int(s) else \
                torch.cuda.default_stream(self.device)
        ctx = torch.cuda.stream(s)
        ctx.__enter__()
        self.guards += (ctx,)
        return s.cuda_stream

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def row_stride(t, name: str, lead, cols: int) -> int:
    """Elements between the rows of ``t`` [*lead, cols], whose rows lie at a uniform
    distance (a contiguous tensor, or columns of one)."""
    check(t.dim() == len(lead) + 1 and t.shape[-1] == cols and tuple(t.shape[:-1]) == tuple(lead),
          f"{name} must be {[*lead, cols]}")
    if t.is_contiguous():
        return cols
    check(t.stride(-1) == 1 or cols == 1, f"{name}'s last dimension must be contiguous")
    step = want = None
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if step is None:
            step, want = stride, stride * size
        else:
            check(stride == want, f"{name}'s rows must lie at one distance")
            want *= size
    if step is None or t.numel() == 0:
        return cols
    check(step >= cols, f"{name}'s rows must not overlap")
    return step


def on_gpu(dtype, device, **tensors):
    """Every given tensor on ``device`` with ``dtype``."""
    for name, t in tensors.items():
        if t is not None:
            check(t.dtype == dtype and t.device == device, f"{name} must be {dtype} on {device}")


def shaped(shape, **tensors):
    """Every given tensor contiguous and of ``shape``."""
    for name, t in tensors.items():
        if t is not None:
            check(t.shape == shape and t.is_contiguous(),
                  f"{name} must be contiguous {list(shape)}")


def io_flags(dtype, out_dtype) -> int:
    if dtype == torch.float32:
        check(out_dtype == torch.float32, "fp32 inputs give fp32 results")
        return GLA_FLAG_FP32_IO
    check(dtype == torch.bfloat16, "inputs must be bf16 or fp32")
    if out_dtype == torch.float32:
        return GLA_FLAG_FP32_OUT
    check(out_dtype == torch.bfloat16, "results come in the inputs' dtype, or fp32")
    return 0


def batch(x, cu_seqlens, name: str):
    """(lead, B, T) of a dense [B, T, cols] or packed [1, R, cols] / [R, cols] tensor."""
    if cu_seqlens is None:
        check(x.dim() == 3, f"a dense {name} is [B, T, D]")
        return x.shape[:2], x.shape[0], x.shape[1]
    check(x.dim() == 2 or (x.dim() == 3 and x.shape[0] == 1),
          f"a packed {name} is [1, R, D] or [R, D]")
    check(cu_seqlens.dtype == torch.int32 and cu_seqlens.device == x.device and
          cu_seqlens.dim() == 1 and cu_seqlens.is_contiguous() and cu_seqlens.numel() >= 2,
          "cu_seqlens must be contiguous int32 [B + 1] on the inputs' GPU")
    return x.shape[:-1], cu_seqlens.numel() - 1, x.shape[-2]


def page_tables(n, device, slots, out_slots):
    for name, t in (("slots", slots), ("out_slots", out_slots)):
        if t is not None:
            check(t.dtype == torch.int32 and t.device == device and t.shape == (n,) and
                  t.is_contiguous(), f"{name} must be contiguous int32 [{n}] on the inputs' GPU")
    check(slots is not None or out_slots is None, "out_slots needs slots")


def scratch(size: int, workspace, device):
    """The given workspace, or a fresh one, of at least ``size`` bytes."""
    if workspace is not None:
        check(workspace.device == device and workspace.dtype == torch.uint8 and
              workspace.is_contiguous() and workspace.data_ptr() % 256 == 0,
              "workspace must be a contiguous, 256-byte aligned uint8 tensor on the inputs' GPU")
        if workspace.numel() >= size:
            return workspace
    return torch.empty(size, dtype=torch.uint8, device=device) if size else None


def done(rc: int, name: str):
    if rc != 0:
        raise GlaError(rc, name)


lib = _binding.lib
