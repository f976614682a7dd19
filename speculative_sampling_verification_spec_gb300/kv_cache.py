"""The paged 8-bit key/value cache of the target's verification pass: append and attention.

`PagedKVCache` describes a pool of pages (e4m3 codes and one float32 scale for each page and key/value head);
`spec_kv_append` and `spec_kv_attention` have the names of the C entry points they call (include/spec_kv.h) and, like
the rest of the binding, only turn torch CUDA tensors into pointers, strides and a stream handle.  There is no CPU or
PyTorch fallback.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import binding

EXPORTED = ("spec_kv_append", "spec_kv_attention", "spec_kv_attention_workspace_size", "spec_kv_capture_id")

# spec_kv_cache and spec_kv_params of include/spec_kv.h, in native layout
_CACHE = struct.Struct("@4i4P5q")
_PARAMS = struct.Struct("@6if3i3P13q3PN")
_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
_DTYPES = {_F32: binding.SPEC_F32, _BF16: binding.SPEC_BF16}
_CODES = (torch.uint8, torch.float8_e4m3fn)
_WS_LEAST = 1 << 20     # bytes of a stream's first workspace: most shapes' later calls need no other


_loaded = None


def _lib():
    global _loaded
    if _loaded is None:
        L = binding.lib()
        P = ctypes.c_void_p
        L.spec_kv_attention_workspace_size.argtypes = [P, P]
        L.spec_kv_attention_workspace_size.restype = ctypes.c_size_t
        L.spec_kv_attention.argtypes = [P] * 5
        L.spec_kv_attention.restype = ctypes.c_int
        L.spec_kv_append.argtypes = [P] * 7
        L.spec_kv_append.restype = ctypes.c_int
        L.spec_kv_capture_id.argtypes = [P]
        L.spec_kv_capture_id.restype = ctypes.c_uint64
        _loaded = L
    return _loaded


class PagedKVCache:
    """A pool of pages: k_codes, v_codes [num_pages, kv_heads, page_size, head_dim] (float8_e4m3fn or uint8; any
    strides that are multiples of 16, channels contiguous, the same for both) and k_scale, v_scale
    [num_pages, kv_heads] float32 (any strides, the same for both).  The tensors are the caller's; the object holds
    their addresses, so it is made once and kept while they live."""

    def __init__(self, k_codes, v_codes, k_scale, v_scale):
        for t in (k_codes, v_codes):
            if t.dim() != 4 or t.dtype not in _CODES or not t.is_cuda:
                raise ValueError("codes must be CUDA float8_e4m3fn or uint8 [num_pages, kv_heads, page_size, head_dim]")
            if t.stride(3) != 1:
                raise ValueError("codes must be contiguous along the channels")
        for t in (k_scale, v_scale):
            if t.dim() != 2 or t.dtype != torch.float32 or not t.is_cuda or t.shape != k_codes.shape[:2]:
                raise ValueError("scales must be CUDA float32 [num_pages, kv_heads]")
        if k_codes.shape != v_codes.shape or k_codes.stride() != v_codes.stride() or \
                k_scale.stride() != v_scale.stride():
            raise ValueError("keys and values must have the same shapes and strides")
        if len({t.device for t in (k_codes, v_codes, k_scale, v_scale)}) != 1:
            raise ValueError("codes and scales must be on one device")
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = k_codes.shape
        self.device = k_codes.device
        self._index = k_codes.get_device()
        st = k_codes.stride()
        self._packed = _CACHE.pack(self.num_pages, self.page_size, self.kv_heads, self.head_dim, k_codes.data_ptr(),
                                   v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), st[0], st[1], st[2],
                                   *k_scale.stride())

    @classmethod
    def empty(cls, num_pages, page_size, kv_heads, head_dim, device="cuda"):
        """A pool with nothing stored (codes and scales are zero)."""
        def codes():
            return torch.zeros((num_pages, kv_heads, page_size, head_dim), dtype=torch.uint8,
                               device=device).view(torch.float8_e4m3fn)
        scales = [torch.zeros((num_pages, kv_heads), dtype=torch.float32, device=device) for _ in range(2)]
        return cls(codes(), codes(), *scales)

    def nbytes(self):
        return sum(t.numel() * t.element_size() for t in (self.k_codes, self.v_codes, self.k_scale, self.v_scale))


# the current stream's handle without building a Stream object, where torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _check_stream(stream, device):
    if stream is not None and stream.device != device:
        raise ValueError("stream is on %s, the cache on %s" % (stream.device, device))


def _stream_of(stream, device):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _new(shape, dtype, device, stream):
    """An output for the call's stream.  One made for another stream than the current one comes from that stream's
    memory, and is recorded on the current one, where the caller goes on to use it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


_ws_cache = {}     # (device, stream) -> workspace
_ws_graphs = {}    # (device, stream) -> (capture, workspace) of the newest capture
_COUNTERS = 1 << 16     # leading bytes that have to be zero before the first use; calls leave them at zero


def _workspace(key, nbytes, device, stream, capture):
    """A workspace of at least nbytes for the calls of one (device, stream): calls on different streams may overlap, so
    each stream has its own.  So has each capture, because graphs are replayed on any stream and may overlap what runs on
    the one they were captured on: the calls of a capture share one from the graph's memory, cleared at every replay."""
    if capture:
        newest = _ws_graphs.get(key)
        if newest is not None and newest[0] == capture and newest[1].numel() >= nbytes:
            return newest[1]
    elif key in _ws_cache:
        nbytes = max(nbytes, 2 * _ws_cache[key].numel())
    with torch.cuda.stream(stream):
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        ws[:_COUNTERS].zero_()
    if capture:
        _ws_graphs[key] = (capture, ws)
    else:
        _ws_cache[key] = ws
    return ws


def spec_kv_reset_workspaces():
    """Forget the workspaces that spec_kv_attention keeps for its callers, so that the next calls start from cleared
    ones: to be called after a SPEC_ERR_TIMEOUT in a status word, which leaves the counters of the call's workspace
    undefined.  (A captured graph clears its own at every replay; a caller's ws is the caller's to clear.)"""
    _ws_cache.clear()
    _ws_graphs.clear()


def _check_table(cache, B, page_table, seq_lens, new_lens, status):
    """The columns and row stride of the page table, after checking it and the lengths."""
    dev = cache._index
    shape = page_table.shape
    if page_table.dtype is not _I32 or len(shape) != 2 or shape[0] != B or shape[1] < 1 or \
            page_table.get_device() != dev:
        raise ValueError("page_table must be int32 [B, max_pages] on the cache's device")
    row, col = page_table.stride()
    if col != 1:
        raise ValueError("page_table must be contiguous along the pages")
    if seq_lens.dtype is not _I32 or seq_lens.shape != (B,) or not seq_lens.is_contiguous() or \
            seq_lens.get_device() != dev:
        raise ValueError("seq_lens must be contiguous int32 [B] on the cache's device")
    if new_lens is not None and (new_lens.dtype is not _I32 or new_lens.shape != (B,) or
                                 not new_lens.is_contiguous() or new_lens.get_device() != dev):
        raise ValueError("new_lens must be contiguous int32 [B] on the cache's device")
    if status is not None and (status.dtype is not _I32 or status.get_device() != dev or status.numel() < 1):
        raise ValueError("status must be int32 [1] on the cache's device")
    return shape[1], row


def _strides(name, t, shape, dtype, device):
    """The strides of a [B, T, heads, head_dim] tensor, after checking it."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        raise ValueError("%s must be %s %s on device %d, got %s %s on %s" % (name, dtype, tuple(shape), device, t.dtype,
                                                                            tuple(t.shape), t.device))
    st = t.stride()
    if st[3] != 1:
        raise ValueError("%s must be contiguous along the channels" % name)
    return st


def _first_check(name, t, heads):
    """Device, type and shape of the tensor that gives a call its sizes."""
    if not t.is_cuda:
        raise ValueError("spec_* calls take CUDA tensors (copy host data to the GPU first)")
    dtype = _DTYPES.get(t.dtype)
    if dtype is None:
        raise TypeError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))
    if t.dim() != 4:
        raise ValueError("%s must be [B, T, %s, head_dim]" % (name, heads))
    return dtype


def spec_kv_append(q, k, v, cache, page_table, seq_lens, new_lens=None, *, cos_sin=None, interleaved=False,
                   q_out=None, status=None, stream=None):
    """Rotate the new tokens' queries and keys by position and store their keys and values.

    q [B, T, Hq, D] (or None), k and v [B, T, kv_heads, D]: float32 or bfloat16, any strides with the channels
    contiguous.  page_table int32 [B, max_pages]; seq_lens int32 [B]: tokens stored before; new_lens int32 [B]: new
    tokens, at most T (None: T each).  cos_sin float32 [positions, rot_dim]: cosines of a position's angles, then their
    sines (None: no rotation); interleaved: pairs are neighbouring channels, else channels i and i + rot_dim / 2.
    Returns the rotated queries (q_out, or a new contiguous tensor; zero in slots past new_lens); q_out may be q.
    The cache is written in place.  The call runs on the cache's device, whichever is current."""
    if _current_device() != cache._index:
        with torch.cuda.device(cache._index):
            return spec_kv_append(q, k, v, cache, page_table, seq_lens, new_lens, cos_sin=cos_sin,
                                  interleaved=interleaved, q_out=q_out, status=status, stream=stream)
    _check_stream(stream, cache.device)
    dtype = _first_check("k", k, "kv_heads")
    shape, dt, dev, index = k.shape, k.dtype, cache.device, cache._index
    B, T, hq, D = shape
    if hq != cache.kv_heads or D != cache.head_dim:
        raise ValueError("k must be [B, T, %d, %d], got %s" % (cache.kv_heads, cache.head_dim, tuple(shape)))
    ks = _strides("k", k, shape, dt, index)
    vs = _strides("v", v, shape, dt, index)
    columns, row = _check_table(cache, B, page_table, seq_lens, new_lens, status)
    rot = rot_len = cs = 0
    if cos_sin is not None:
        if cos_sin.dtype is not _F32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous() or cos_sin.get_device() != index:
            raise ValueError("cos_sin must be contiguous float32 [positions, rot_dim] on the cache's device")
        rot_len, rot = cos_sin.shape
        cs = cos_sin.data_ptr()
    qs, os, qp, op = (0, 0, 0, 1), (0, 0, 0, 1), 0, 0
    if q is not None:
        if q.dim() != 4:
            raise ValueError("q must be [B, T, Hq, head_dim]")
        hq = q.shape[2]
        shape = (B, T, hq, D)
        qs = _strides("q", q, shape, dt, index)
        if q_out is None:
            q_out = _new(shape, dt, dev, stream)
            os = q_out.stride()
        else:
            os = _strides("q_out", q_out, shape, dt, index)
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    prm = _PARAMS.pack(B, T, hq, dtype, columns, 0, 0.0, rot, rot_len, 1 if interleaved else 0,
                       page_table.data_ptr(), seq_lens.data_ptr(), 0 if new_lens is None else new_lens.data_ptr(),
                       row, qs[0], qs[1], qs[2], ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], os[0],
                       os[1], os[2], _stream_of(stream, dev), 0 if status is None else status.data_ptr(), 0, 0)
    code = _lib().spec_kv_append(qp, k.data_ptr(), v.data_ptr(), cs, cache._packed, prm, op)
    if code != binding.SPEC_OK:
        raise binding.SpecError(code, "spec_kv_append")
    return q_out


def spec_kv_attention(q, cache, page_table, seq_lens, new_lens=None, *, scale=None, window=0, out=None, lse=None,
                      return_lse=False, status=None, ws=None, stream=None):
    """Attention of the new tokens' (rotated) queries over everything stored for their sequence up to themselves.

    q [B, T, Hq, D] float32 or bfloat16; page_table, seq_lens and new_lens as for the spec_kv_append that stored the
    new tokens.  scale: factor of the scores (1 / sqrt(D)); window > 0: a query sees that many tokens, its own
    included.  Returns out [B, T, Hq, D] (zero in slots past new_lens), or (out, lse) with lse [B, T, Hq] float32, the
    natural logarithm of the sum of the weights, when return_lse or lse is given.  ws: a workspace of
    spec_kv_attention_workspace_size bytes (uint8, CUDA, zeroed once); by default one is kept for each stream
    and one for each graph that is captured.  The call runs on the cache's device, whichever is current."""
    if _current_device() != cache._index:
        with torch.cuda.device(cache._index):
            return spec_kv_attention(q, cache, page_table, seq_lens, new_lens, scale=scale, window=window, out=out,
                                     lse=lse, return_lse=return_lse, status=status, ws=ws, stream=stream)
    _check_stream(stream, cache.device)
    dtype = _first_check("q", q, "Hq")
    shape, dt, dev, index = q.shape, q.dtype, cache.device, cache._index
    B, T, hq, D = shape
    if D != cache.head_dim:
        raise ValueError("q must be [B, T, Hq, %d], got %s" % (cache.head_dim, tuple(shape)))
    qs = _strides("q", q, shape, dt, index)
    columns, row = _check_table(cache, B, page_table, seq_lens, new_lens, status)
    if out is None:
        out = _new(shape, dt, dev, stream)
        os = out.stride()
    else:
        os = _strides("out", out, shape, dt, index)
    if lse is not None:
        if lse.dtype is not _F32 or lse.shape != shape[:3] or not lse.is_contiguous() or lse.get_device() != index:
            raise ValueError("lse must be contiguous float32 [B, T, Hq] on the cache's device")
    elif return_lse:
        lse = _new(shape[:3], _F32, dev, stream)
    handle = _stream_of(stream, dev)
    key = (index, handle)
    L = _lib()
    capture = own = 0
    if ws is None:
        own = 1
        # (asked of torch where it is about the current stream, which is cheaper)
        if stream is not None or torch.cuda.is_current_stream_capturing():
            capture = L.spec_kv_capture_id(handle)
        if not capture:
            ws = _ws_cache.get(key)
    elif ws.dtype is not torch.uint8 or ws.get_device() != index or not ws.is_contiguous():
        raise ValueError("ws must be contiguous uint8 on the cache's device")
    fixed = (B, T, hq, dtype, columns, window, 1.0 / math.sqrt(D) if scale is None else scale, 0, 0, 0,
             page_table.data_ptr(), seq_lens.data_ptr(), 0 if new_lens is None else new_lens.data_ptr(),
             row, qs[0], qs[1], qs[2], 0, 0, 0, 0, 0, 0, os[0], os[1], os[2], handle,
             0 if status is None else status.data_ptr())
    args = (q.data_ptr(), cache._packed, out.data_ptr(), 0 if lse is None else lse.data_ptr())
    if ws is None:
        nbytes = L.spec_kv_attention_workspace_size(cache._packed, _PARAMS.pack(*fixed, 0, 0))
        ws = _workspace(key, max(nbytes, _WS_LEAST), dev, stream, capture)
    code = L.spec_kv_attention(args[0], args[1], _PARAMS.pack(*fixed, ws.data_ptr(), ws.numel()), args[2], args[3])
    if code == binding.SPEC_ERR_INVALID_ARG and own and not capture:
        # the stream's workspace may be too small for this shape: a larger one is made, once
        nbytes = L.spec_kv_attention_workspace_size(cache._packed, _PARAMS.pack(*fixed, 0, 0))
        if nbytes > ws.numel():
            ws = _workspace(key, nbytes, dev, stream, capture)
            code = L.spec_kv_attention(args[0], args[1], _PARAMS.pack(*fixed, ws.data_ptr(), ws.numel()), args[2],
                                       args[3])
    if code != binding.SPEC_OK:
        raise binding.SpecError(code, "spec_kv_attention")
    return out if lse is None else (out, lse)


def spec_kv_attention_workspace_size(cache, B, T, Hq, dtype=torch.bfloat16) -> int:
    """Workspace bytes of a spec_kv_attention call of this shape (0 if it is invalid)."""
    prm = _PARAMS.pack(B, T, Hq, _DTYPES.get(dtype, -1), 1, 0, 1.0, 0, 0, 0, 0, 0, 0, *([0] * 13), 0, 0, 0, 0)
    return int(_lib().spec_kv_attention_workspace_size(cache._packed, prm))
