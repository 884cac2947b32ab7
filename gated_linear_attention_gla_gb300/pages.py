"""The pages of state pools (argument marshalling only).

A sequence's recurrent state is one page, under one number, in every pool of a
model: fp32 [num_pages, H, dk, dv] for ``decode_step``, [num_pages, W - 1, D] for
``conv_step``, fp32 [num_pages, D, N] for ``scan_step``, one pool per layer.
``used`` (int32 [num_pages] on the GPU, 0 = free) says which pages are taken.
The functions below read and write such tables on the GPU and move the pages of
all given pools; nothing waits for the host, and they can be captured into CUDA
graphs.  Bad entries are skipped and raise in the next ``status_sync``.
"""
from __future__ import annotations

from typing import Sequence

import torch

from ._binding import GLA_PAGE_NEW, PagePool
from ._marshal import check, done, launch_on, lib, ptr

PAGE_NEW = GLA_PAGE_NEW  # a parent for fork_pages: a page of zeros


def _table(t, name: str, device=None, n=None):
    if not t.is_cuda or t.dtype is not torch.int32 or t.dim() != 1 or not t.is_contiguous() or \
            (device is not None and t.device != device) or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must be contiguous int32 [{'n' if n is None else n}] on the "
                         "pools' GPU")
    return t


def _pools(pools: Sequence[torch.Tensor], device, pages=None):
    """(C array of the pools, their number, their pages)."""
    if isinstance(pools, torch.Tensor):
        pools = (pools,)
    arr = (PagePool * max(1, len(pools)))()
    for i, p in enumerate(pools):
        check(p.device == device and p.is_contiguous() and p.dim() >= 2,
              "a pool must be a contiguous tensor [num_pages, ...] on the tables' GPU")
        n = p.shape[0]
        pages = n if pages is None else pages
        check(n == pages, "the pools and the table have one number of pages")
        arr[i] = PagePool(p.data_ptr(), p.numel() // max(1, n) * p.element_size())
    return arr, len(pools) if pages else 0, pages or 0


def copy_pages(pools, src, dst, copied=None, stream=None):
    """Page ``dst[i]`` = page ``src[i]`` in every pool, for all pairs at once (int32 [n];
    -1 skips).  Pairs whose dst another pair writes or reads are skipped and
    reported.  Returns ``copied`` [n]: dst[i] where it was copied, else -1."""
    dev = _table(src, "src").device
    n = src.shape[0]
    _table(dst, "dst", dev, n)
    arr, count, pages = _pools(pools, dev)
    with launch_on(dev, stream) as s:
        copied = torch.empty_like(src) if copied is None else _table(copied, "copied", dev, n)
        done(lib().gla_pages_copy(arr, count, pages, ptr(src), ptr(dst), ptr(copied), n, s),
             "gla_pages_copy")
    return copied


def fork_pages(pools, used, parents, children=None, used_out=None, stream=None):
    """A new page for every entry of ``parents`` (int32 [n]): a copy of page parents[i] in
    every pool, zeros for PAGE_NEW, none for -1.  The free pages in ascending
    order go to the entries in order; -1 (and a report) when none is left.
    Returns ``(children, used_out)``; ``used`` is updated in place unless
    ``used_out`` is given."""
    dev = _table(used, "used").device
    n = _table(parents, "parents", dev).shape[0]
    arr, count, pages = _pools(pools, dev, used.shape[0])
    used_out = used if used_out is None else _table(used_out, "used_out", dev, pages)
    with launch_on(dev, stream) as s:
        children = torch.empty_like(parents) if children is None else \
            _table(children, "children", dev, n)
        done(lib().gla_pages_fork(arr, count, pages, ptr(used), ptr(used_out), ptr(parents),
                                  ptr(children), n, s), "gla_pages_fork")
    return children, used_out


def compact_pages(pools, used, slots, slots_out=None, used_out=None, forward=None, stream=None):
    """Moves the used pages to the front of every pool: with L pages used, those at or
    behind L go to the free pages in front of L, in ascending order.  Returns
    ``(slots_out, used_out, forward)``: ``slots`` (int32 [n], -1 stays) with the
    new numbers, the table, and every page's new number (-1: free).  ``used`` is
    updated in place unless ``used_out`` is given; ``slots_out`` is a new tensor
    unless given (it may be ``slots``)."""
    dev = _table(used, "used").device
    n = _table(slots, "slots", dev).shape[0]
    arr, count, pages = _pools(pools, dev, used.shape[0])
    used_out = used if used_out is None else _table(used_out, "used_out", dev, pages)
    with launch_on(dev, stream) as s:
        slots_out = torch.empty_like(slots) if slots_out is None else \
            _table(slots_out, "slots_out", dev, n)
        forward = torch.empty_like(used) if forward is None else \
            _table(forward, "forward", dev, pages)
        done(lib().gla_pages_compact(arr, count, pages, ptr(used), ptr(used_out), ptr(slots),
                                     ptr(slots_out), n, ptr(forward), s), "gla_pages_compact")
    return slots_out, used_out, forward


def free_pages(used, slots, used_out=None, stream=None):
    """Marks the pages ``slots`` (int32 [n], -1 skips) free; their contents stay.  Returns
    the table (``used`` itself unless ``used_out`` is given)."""
    dev = _table(used, "used").device
    n = _table(slots, "slots", dev).shape[0]
    used_out = used if used_out is None else _table(used_out, "used_out", dev, used.shape[0])
    with launch_on(dev, stream) as s:
        done(lib().gla_pages_free(ptr(used), ptr(used_out), used.shape[0], ptr(slots), n, s),
             "gla_pages_free")
    return used_out
