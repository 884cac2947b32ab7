"""Argument marshalling shared by ``ssm``, ``block`` and ``pages``: checks, row strides,
the device and stream a call runs on."""
from __future__ import annotations

import torch

from . import _binding
from ._binding import GLA_FLAG_FP32_IO, GLA_FLAG_FP32_OUT, GlaError


# The current device and stream as plain ints, without building objects (the
# decode paths are a few microseconds of kernel).
_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else \
    torch.cuda.current_device
_stream = torch._C._cuda_getCurrentRawStream \
    if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    lambda index: torch.cuda.current_stream(index).cuda_stream


def check(cond: bool, msg: str):
    """For constant messages; a message that has to be formed is raised in place, so
    that calls which are fine do not pay for it."""
    if not cond:
        raise ValueError(msg)


def counted(n: int, what: str) -> int:
    """A number of rows, sequences, channels or pages as the library takes it, a C int (ctypes cuts
    off what does not fit)."""
    if n > 0x7fffffff:
        raise ValueError(f"{n} {what}: at most 2^31 - 1")
    return n


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
        index = self.device.index
        if index != _device():
            self.guards = (torch.cuda.device(self.device),)
            self.guards[0].__enter__()
        if self.stream is None:
            return _stream(index)
        s = self.stream
        if not isinstance(s, torch.cuda.Stream):
            s = torch.cuda.ExternalStream(int(s), device=self.device) if int(s) else \
                torch.cuda.default_stream(self.device)
        if s.device != self.device:
            self.__exit__()
            raise ValueError(f"the stream is on {s.device}, the tensors on {self.device}")
        ctx = torch.cuda.stream(s)
        ctx.__enter__()
        self.guards += (ctx,)
        return s.cuda_stream

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc or (None, None, None))


def rows(t, name: str, shape, dtype, device):
    """(address, elements between rows) of ``t``, of ``shape`` [*lead, cols], whose rows lie
    at a uniform distance (a contiguous tensor, or columns of one)."""
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        raise ValueError(f"{name} must be {dtype} {list(shape)} on {device}")
    st, n, cols = t.stride(), len(shape), shape[-1]
    if st[-1] != 1 and cols != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    if n == 2:
        step = st[0] if shape[0] > 1 else None
    elif n == 3 and shape[1] > 1:
        step = st[1]
        if shape[0] > 1 and st[0] != step * shape[1]:
            raise ValueError(f"{name}'s rows must lie at one distance")
    elif n == 3:
        step = st[0] if shape[0] > 1 else None
    else:
        raise ValueError(f"{name} must have two or three dimensions")
    if step is None or t.numel() == 0:
        return t.data_ptr(), cols
    if step < cols:
        raise ValueError(f"{name}'s rows must not overlap")
    return t.data_ptr(), step


def whole(t, name: str, shape, dtype, device):
    """The address of ``t`` (None: 0), contiguous and of ``shape``."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)} on {device}")
    return t.data_ptr()


def io_flags(dtype, out_dtype) -> int:
    if dtype is torch.float32:
        check(out_dtype is torch.float32, "fp32 inputs give fp32 results")
        return GLA_FLAG_FP32_IO
    check(dtype is torch.bfloat16, "inputs must be bf16 or fp32")
    if out_dtype is torch.float32:
        return GLA_FLAG_FP32_OUT
    check(out_dtype is torch.bfloat16, "results come in the inputs' dtype, or fp32")
    return 0


def batch(x, cu_seqlens, name: str):
    """(lead, B, T) of a dense [B, T, cols] or packed [1, R, cols] / [R, cols] tensor."""
    if cu_seqlens is None:
        if x.dim() != 3:
            raise ValueError(f"a dense {name} is [B, T, D]")
        lead = x.shape[:2]
        return lead, counted(lead[0], "sequences"), counted(lead[1], "tokens")
    if x.dim() != 2 and not (x.dim() == 3 and x.shape[0] == 1):
        raise ValueError(f"a packed {name} is [1, R, D] or [R, D]")
    check(cu_seqlens.dtype is torch.int32 and cu_seqlens.device == x.device and
          cu_seqlens.dim() == 1 and cu_seqlens.is_contiguous() and cu_seqlens.numel() >= 2,
          "cu_seqlens must be contiguous int32 [B + 1] on the inputs' GPU")
    return x.shape[:-1], counted(cu_seqlens.numel() - 1, "sequences"), counted(x.shape[-2], "rows")


def output(out, shape, dtype, device):
    """The given output, checked, or a fresh one."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if out.shape != shape or not out.is_contiguous() or out.device != device:
        raise ValueError(f"out must be contiguous {list(shape)} on {device}")
    return out


def page_tables(n, device, slots, out_slots):
    """The addresses of the tables of pages read and written."""
    if slots is None:
        check(out_slots is None, "out_slots needs slots")
        return None, None
    return (whole(slots, "slots", (n,), torch.int32, device),
            whole(out_slots, "out_slots", (n,), torch.int32, device))


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
