"""Who holds the pages of a paged key/value cache: holding and forking.

`spec_kv_hold` and `spec_kv_fork` have the names of the C entry points they call (include/spec_kv_pages.h) and only turn
torch CUDA tensors into pointers, strides and a stream handle.  The page table and the counts of the pages' holders are
the caller's tensors and are written in place, on the device: an empty pool is a table of -1 and counts of 0.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import binding
from .kv_cache import _check_stream, _current_device, _stream_of

EXPORTED = ("spec_kv_fork", "spec_kv_hold")

# spec_kv_pages of include/spec_kv_pages.h, in native layout
_PAGES = struct.Struct("@4i2Pq3P")
_I32 = torch.int32
_MOST_INT = (1 << 31) - 1     # (ctypes would drop the bits above, of negative ones too)

_loaded = None


def _lib():
    global _loaded
    if _loaded is None:
        L = binding.lib()
        P, I = ctypes.c_void_p, ctypes.c_int32
        L.spec_kv_hold.argtypes = [P, P, P, I, I, I]
        L.spec_kv_hold.restype = ctypes.c_int
        L.spec_kv_fork.argtypes = [P, P, P, P]
        L.spec_kv_fork.restype = ctypes.c_int
        _loaded = L
    return _loaded


def _check(name, t, B, device):
    if t.dtype is not _I32 or t.shape != (B,) or not t.is_contiguous() or t.get_device() != device:
        raise ValueError("%s must be contiguous int32 [B] on the counts' device" % name)
    return t.data_ptr()


def _pages(refs, page_table, page_size, free, status, stream):
    """The packed spec_kv_pages, after checking the tensors."""
    dev = refs.get_device()
    if refs.dtype is not _I32 or refs.dim() != 1 or not refs.is_contiguous():
        raise ValueError("refs must be contiguous int32 [num_pages]")
    shape = page_table.shape
    if page_table.dtype is not _I32 or len(shape) != 2 or shape[1] < 1 or page_table.get_device() != dev:
        raise ValueError("page_table must be int32 [B, max_pages] on the counts' device")
    row, col = page_table.stride()
    if col != 1:
        raise ValueError("page_table must be contiguous along the pages")
    for name, t in (("free", free), ("status", status)):
        if t is not None and (t.dtype is not _I32 or t.get_device() != dev or t.numel() < 1):
            raise ValueError("%s must be int32 [1] on the counts' device" % name)
    return _PAGES.pack(refs.shape[0], page_size, shape[0], shape[1], refs.data_ptr(), page_table.data_ptr(), row,
                       0 if free is None else free.data_ptr(), _stream_of(stream, refs.device),
                       0 if status is None else status.data_ptr())


def _on_device(refs, stream):
    if not refs.is_cuda:
        raise ValueError("spec_* calls take CUDA tensors (copy host data to the GPU first)")
    _check_stream(stream, refs.device)
    return _current_device() == refs.get_device()


def spec_kv_hold(refs, page_table, seq_lens, new_lens=None, *, page_size, T=0, window=0, sinks=0, free=None, status=None,
                 stream=None):
    """Give each sequence exactly the pages that its tokens need: take free ones for what is missing, release the others.

    refs int32 [num_pages]: table entries that hold each page (0: free); page_table int32 [B, max_pages], -1 where none;
    seq_lens int32 [B]: tokens stored; new_lens int32 [B]: tokens to come (None: T each).  With a window, pages before the
    last window - 1 stored tokens are released, but for those of the first `sinks` ones.  refs and page_table are written
    in place; free int32 [1], when given, gets the number of free pages left.  Where they do not suffice, the last entries
    stay negative, with SPEC_ERR_CACHE_FULL in status.  The call runs on the counts' device, whichever is current."""
    if not _on_device(refs, stream):
        with torch.cuda.device(refs.device):
            return spec_kv_hold(refs, page_table, seq_lens, new_lens, page_size=page_size, T=T, window=window, sinks=sinks,
                                free=free, status=status, stream=stream)
    if min(T, window, sinks) < 0 or max(T, window, sinks, page_size) > _MOST_INT:
        raise binding.SpecError(binding.SPEC_ERR_INVALID_ARG, "spec_kv_hold")
    pages = _pages(refs, page_table, page_size, free, status, stream)
    B, dev = page_table.shape[0], refs.get_device()
    code = _lib().spec_kv_hold(pages, _check("seq_lens", seq_lens, B, dev),
                               None if new_lens is None else _check("new_lens", new_lens, B, dev), T, window, sinks)
    if code != binding.SPEC_OK:
        raise binding.SpecError(code, "spec_kv_hold")


def spec_kv_fork(cache, refs, page_table, seq_lens, parents, *, free=None, status=None, stream=None):
    """Make sequences copies of others: parents int32 [B] has the sequence that each becomes a copy of, or -1 (or its own
    number) where it stays, as every parent has to.  Whole pages are shared, the last one, partly filled, is copied to a
    free page, and what a copy held before is released.

    cache: the PagedKVCache; refs, page_table, seq_lens as for spec_kv_hold, written in place; free, status likewise.  The
    call runs on the cache's device, whichever is current."""
    if not _on_device(refs, stream):
        with torch.cuda.device(refs.device):
            return spec_kv_fork(cache, refs, page_table, seq_lens, parents, free=free, status=status, stream=stream)
    if refs.device != cache.device or refs.shape != (cache.num_pages,):
        raise ValueError("refs must be int32 [num_pages] on the cache's device")
    pages = _pages(refs, page_table, cache.page_size, free, status, stream)
    B, dev = page_table.shape[0], refs.get_device()
    code = _lib().spec_kv_fork(pages, cache._packed, _check("seq_lens", seq_lens, B, dev),
                               _check("parents", parents, B, dev))
    if code != binding.SPEC_OK:
        raise binding.SpecError(code, "spec_kv_fork")
