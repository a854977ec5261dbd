"""Paged key cache: rows written (quantised) at their slots, read back at positions, attended to.

Python face of ``include/sel/cache.h``, in the manner of the package's top-k and gather: PyTorch supplies
device memory and the stream, every step of the computation runs in the library's kernels, argument errors
raise before a launch, findings made on the device go to a caller-zeroed ``err_flag``.

A cache is ``[pages, page_size, d]``: bf16 rows, or ``torch.float8_e4m3fn`` codes with ``scales`` fp32
``[pages, page_size, ceil(d / 128)]`` (value = code * scale; ``cache_write`` stores powers of two).  One row a
position, shared by all heads.  ``page_table`` int32 ``[b, max_pages]`` lists each sequence's pages; row r of a
call belongs to sequence ``r // (rows // b)``.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from . import _native

GROUP = _native.SEL_CACHE_GROUP
_IDX = {torch.int32: _native.SEL_I32, torch.int64: _native.SEL_I64}
_ROWS = {torch.float32: _native.SEL_F32, torch.bfloat16: _native.SEL_BF16}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _flag(err_flag, dev):
    if err_flag is not None and (err_flag.dtype != torch.int32 or err_flag.numel() < 1 or err_flag.device != dev):
        raise ValueError("err_flag must be an int32 tensor on the cache's device")
    return _ptr(err_flag)


def _cache_struct(cache, scales):
    """The C struct of a cache, and the tensors' checks."""
    if cache.dim() != 3 or cache.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
        raise ValueError("cache must be a 3-D bfloat16 or float8_e4m3fn tensor [pages, page_size, d]")
    if not cache.is_cuda:
        raise ValueError("cache must be a CUDA tensor")
    pages, page_size, d = cache.shape
    if d > 1 and cache.stride(2) != 1:
        raise ValueError("cache rows must be contiguous in their last dimension")
    c = _native.SelCache()
    c.data = cache.data_ptr()
    c.pages, c.page_size, c.d = pages, page_size, d
    c.row_stride = cache.stride(1) if page_size > 1 else d
    c.page_stride = cache.stride(0) if pages > 1 else page_size * c.row_stride
    if cache.dtype == torch.bfloat16:
        if scales is not None:
            raise ValueError("a bfloat16 cache has no scales")
        c.dtype = _native.SEL_BF16
        return c
    c.dtype = _native.SEL_E4M3
    runs = -(-d // GROUP)
    if scales is None or scales.dtype != torch.float32 or tuple(scales.shape) != (pages, page_size, runs) \
            or scales.device != cache.device:
        raise ValueError("a float8_e4m3fn cache needs float32 scales [pages, page_size, ceil(d / %d)] on its device"
                         % GROUP)
    if runs > 1 and scales.stride(2) != 1:
        raise ValueError("scales must be contiguous in their last dimension")
    c.scales = scales.data_ptr()
    c.scale_row_stride = scales.stride(1) if page_size > 1 else runs
    c.scale_page_stride = scales.stride(0) if pages > 1 else page_size * c.scale_row_stride
    return c


def _table(page_table, dev):
    if page_table.dim() != 2 or page_table.dtype != torch.int32 or page_table.device != dev:
        raise ValueError("page_table must be an int32 tensor [b, max_pages] on the cache's device")
    if page_table.shape[0] < 1:
        raise ValueError("page_table needs a row for each sequence")
    if page_table.shape[1] > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table rows must be contiguous")
    b, m = page_table.shape
    return b, m, page_table.stride(0) if b > 1 else m


def _index(idx, dev):
    if idx.dim() != 2 or idx.dtype not in _IDX or idx.device != dev:
        raise ValueError("idx must be a 2-D int32/int64 tensor on the cache's device")
    if idx.size(1) > 1 and idx.stride(1) != 1:
        raise ValueError("idx rows must be contiguous")
    return idx.stride(0) if idx.size(0) > 1 else idx.size(1)


@contextlib.contextmanager
def _on(dev, stream):
    """The device, and the stream to launch and allocate on (so that outputs and scratch belong to it)."""
    with torch.cuda.device(dev):
        if stream is None:
            yield ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)
        else:
            with torch.cuda.stream(stream):
                yield ctypes.c_void_p(stream.cuda_stream)


def cache_write(x: torch.Tensor, cache: torch.Tensor, slots: torch.Tensor, *, scales: torch.Tensor | None = None,
                err_flag: torch.Tensor | None = None, stream=None) -> None:
    """Writes rows ``x`` [tokens, d] (bf16 or fp32, rows may be strided) into ``cache`` at ``slots``
    (int32/int64 [tokens], slot = page * page_size + row in the page; negative: a padding token, skipped).

    A float8_e4m3fn cache gets, for each run of 128 elements, the smallest power of two that brings the run's
    largest finite magnitude to 448 or less (``scales``) and the values over it, rounded to nearest even; an
    infinity is stored as 448 times the scale, a NaN as NaN.  Slots have to differ; one past the cache writes
    nothing and sets ``err_flag``.
    """
    c = _cache_struct(cache, scales)
    dev = cache.device
    if x.dim() != 2 or x.dtype not in _ROWS or x.device != dev or x.shape[1] != cache.shape[2]:
        raise ValueError("x must be a bfloat16 or float32 tensor [tokens, d] on the cache's device")
    if x.size(1) > 1 and x.stride(1) != 1:
        raise ValueError("rows of x must be contiguous")
    tokens = x.shape[0]
    if slots.dim() != 1 or slots.dtype not in _IDX or slots.numel() != tokens or slots.device != dev \
            or not slots.is_contiguous():
        raise ValueError("slots must be a contiguous int32/int64 tensor with one entry per token")
    err = _flag(err_flag, dev)
    with _on(dev, stream) as s:
        st = _native.load().sel_cache_write(
            _ptr(x), _ROWS[x.dtype], tokens, x.stride(0) if tokens > 1 else x.shape[1], _ptr(slots),
            _IDX[slots.dtype], ctypes.byref(c), err, s)
    _native.check(st, "sel_cache_write")


def cache_gather(cache: torch.Tensor, page_table: torch.Tensor, idx: torch.Tensor, *,
                 scales: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 err_flag: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[r, j, :] = the cache row at position max(idx[r, j], 0) of row r's sequence, as bf16 [rows, n, d].

    idx: int32/int64 [rows, n], rows a multiple of the page table's b.  A position outside the page table or on
    a page outside the cache yields a zero row and sets ``err_flag``.
    """
    c = _cache_struct(cache, scales)
    dev = cache.device
    b, m, ts = _table(page_table, dev)
    irs = _index(idx, dev)
    rows, n = idx.shape
    d = cache.shape[2]
    if out is not None and (out.shape != (rows, n, d) or not out.is_contiguous() or out.dtype != torch.bfloat16
                            or out.device != dev):
        raise ValueError("out must be a contiguous bf16 [rows, n, d] tensor")
    err = _flag(err_flag, dev)
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty((rows, n, d), dtype=torch.bfloat16, device=dev)
        st = _native.load().sel_cache_gather(
            ctypes.byref(c), _ptr(page_table), b, m, ts, _ptr(idx), _IDX[idx.dtype], rows, n, irs, _ptr(out),
            err, s)
    _native.check(st, "sel_cache_gather")
    return out


def cache_attention(q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor, *,
                    scales: torch.Tensor | None = None, end: torch.Tensor | None = None,
                    idx: torch.Tensor | None = None, dv: int | None = None, scale: float | None = None,
                    return_lse: bool = False, out: torch.Tensor | None = None,
                    err_flag: torch.Tensor | None = None, stream=None):
    """Attention of new tokens ``q`` (bf16 [rows, h, d], rows and heads may be strided) over the cache.

    Each row attends to the positions of its sequence below ``end[r]`` (int32 [rows], exclusive; None: the whole
    page table), or, with ``idx`` (int32/int64 [rows, n], a selection's output), to the positions listed there
    (negative: none; at or past ``end``: left out).  Scores are ``scale * <q, row>`` (default 1 / sqrt(d)); the
    value is the row's first ``dv`` elements (default d, at most 512, a multiple of 8).  A row without positions
    gives zeros and a log-sum of -inf.  Positions a row does not attend to never influence it.

    Returns ``(out, lse)``: bf16 [rows, h, dv], and fp32 [rows, h] (natural log of the sum of exponentials) with
    ``return_lse``, else None.
    """
    c = _cache_struct(cache, scales)
    dev = cache.device
    b, m, ts = _table(page_table, dev)
    d = cache.shape[2]
    if q.dim() != 3 or q.dtype != torch.bfloat16 or q.device != dev or q.shape[2] != d:
        raise ValueError("q must be a bfloat16 tensor [rows, h, d] on the cache's device")
    if d > 1 and q.stride(2) != 1:
        raise ValueError("q must be contiguous in its last dimension")
    rows, h, _ = q.shape
    if end is not None and (end.dtype != torch.int32 or end.dim() != 1 or end.numel() != rows or end.device != dev
                            or not end.is_contiguous()):
        raise ValueError("end must be a contiguous int32 tensor with one entry per row")
    dv = d if dv is None else int(dv)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    irs = n = itype = 0
    if idx is not None:
        irs = _index(idx, dev)
        if idx.shape[0] != rows:
            raise ValueError("idx must have one row per row of q")
        n, itype = idx.shape[1], _IDX[idx.dtype]
    if out is not None and (out.shape != (rows, h, dv) or not out.is_contiguous() or out.dtype != torch.bfloat16
                            or out.device != dev):
        raise ValueError("out must be a contiguous bf16 [rows, h, dv] tensor")
    err = _flag(err_flag, dev)
    lib = _native.load()
    # an empty index list has no address of its own: any address says that idx was given
    ip = None if idx is None else (_ptr(idx) if n > 0 else _ptr(page_table) or _ptr(q))
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty((rows, h, max(dv, 0)), dtype=torch.bfloat16, device=dev)
        lse = torch.empty((rows, h), dtype=torch.float32, device=dev) if return_lse else None
        need = int(lib.sel_cache_attention_workspace_size(rows, h, d, dv, b, m, cache.shape[1], int(idx is not None),
                                                          n))
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        st = lib.sel_cache_attention(
            _ptr(q), rows, h, q.stride(0) if rows > 1 else h * d, q.stride(1) if h > 1 else d, ctypes.byref(c),
            _ptr(page_table), b, m, ts, _ptr(end), ip, itype, n, irs, dv, scale, _ptr(out), _ptr(lse), _ptr(ws),
            need, err, s)
    _native.check(st, "sel_cache_attention")
    return out, lse
