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

import functools
import math

import torch

from . import _native

GROUP = _native.SEL_CACHE_GROUP
_IDX = {torch.int32: _native.SEL_I32, torch.int64: _native.SEL_I64}
_ROWS = {torch.float32: _native.SEL_F32, torch.bfloat16: _native.SEL_BF16}


_CACHES = {torch.bfloat16: _native.SEL_BF16, torch.float8_e4m3fn: _native.SEL_E4M3}


def _flag(err_flag, dev):
    if err_flag is None:
        return None
    if err_flag.dtype != torch.int32 or err_flag.numel() < 1 or err_flag.device != dev:
        raise ValueError("err_flag must be an int32 tensor on the cache's device")
    return err_flag.data_ptr()


def _cache_struct(cache, scales):
    """The C struct of a cache, and the tensors' checks."""
    kind = _CACHES.get(cache.dtype)
    if kind is None or cache.dim() != 3:
        raise ValueError("cache must be a 3-D bfloat16 or float8_e4m3fn tensor [pages, page_size, d]")
    if not cache.is_cuda:
        raise ValueError("cache must be a CUDA tensor")
    pages, page_size, d = cache.shape
    page_stride, row_stride, one = cache.stride()
    if one != 1 and d > 1:
        raise ValueError("cache rows must be contiguous in their last dimension")
    if page_size == 1:
        row_stride = d
    if pages == 1:
        page_stride = page_size * row_stride
    if kind == _native.SEL_BF16:
        if scales is not None:
            raise ValueError("a bfloat16 cache has no scales")
        return _native.SelCache(cache.data_ptr(), None, kind, pages, page_size, d, page_stride, row_stride, 0, 0)
    runs = -(-d // GROUP)
    if scales is None or scales.dtype != torch.float32 or scales.shape != (pages, page_size, runs) \
            or scales.device != cache.device:
        raise ValueError("a float8_e4m3fn cache needs float32 scales [pages, page_size, ceil(d / %d)] on its device"
                         % GROUP)
    s_page, s_row, one = scales.stride()
    if one != 1 and runs > 1:
        raise ValueError("scales must be contiguous in their last dimension")
    if page_size == 1:
        s_row = runs
    if pages == 1:
        s_page = page_size * s_row
    return _native.SelCache(cache.data_ptr(), scales.data_ptr(), kind, pages, page_size, d, page_stride, row_stride,
                            s_page, s_row)


def _table(page_table, dev):
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.device != dev:
        raise ValueError("page_table must be an int32 tensor [b, max_pages] on the cache's device")
    b, m = page_table.shape
    if b < 1:
        raise ValueError("page_table needs a row for each sequence")
    stride, one = page_table.stride()
    if one != 1 and m > 1:
        raise ValueError("page_table rows must be contiguous")
    return b, m, stride if b > 1 else m


def _index(idx, dev):
    if idx.dtype not in _IDX or idx.dim() != 2 or idx.device != dev:
        raise ValueError("idx must be a 2-D int32/int64 tensor on the cache's device")
    rows, n = idx.shape
    stride, one = idx.stride()
    if one != 1 and n > 1:
        raise ValueError("idx rows must be contiguous")
    return rows, n, stride if rows > 1 else n


def _launch(dev, stream, call):
    """``call(raw stream)`` with ``dev`` current and, where a stream is given, that stream current too (so that
    what the call allocates belongs to it)."""
    if stream is not None:
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            return call(stream.cuda_stream)
    index = dev.index
    if index == torch.cuda.current_device():  # (the two context managers cost several microseconds)
        return call(torch._C._cuda_getCurrentRawStream(index))
    with torch.cuda.device(dev):
        return call(torch._C._cuda_getCurrentRawStream(index))


@functools.lru_cache(maxsize=4096)
def _scratch_bytes(device_index, rows, h, d, dv, b, max_pages, page_size, idx_given, n):
    """Scratch that a call of this shape needs on the (current) device."""
    return int(_native.load().sel_cache_attention_workspace_size(rows, h, d, dv, b, max_pages, page_size, idx_given,
                                                                 n))


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
    x_type = _ROWS.get(x.dtype)
    if x_type is None or x.dim() != 2 or x.device != dev or x.shape[1] != c.d:
        raise ValueError("x must be a bfloat16 or float32 tensor [tokens, d] on the cache's device")
    tokens, d = x.shape
    x_stride, one = x.stride()
    if one != 1 and d > 1:
        raise ValueError("rows of x must be contiguous")
    slot_type = _IDX.get(slots.dtype)
    if slot_type is None or slots.dim() != 1 or slots.shape[0] != tokens or slots.device != dev \
            or not slots.is_contiguous():
        raise ValueError("slots must be a contiguous int32/int64 tensor with one entry per token")
    err = _flag(err_flag, dev)
    _native.check(_launch(dev, stream, lambda s: _native.load().sel_cache_write(
        x.data_ptr(), x_type, tokens, x_stride if tokens > 1 else d, slots.data_ptr(), slot_type, c, err, s)),
        "sel_cache_write")


def cache_gather(cache: torch.Tensor, page_table: torch.Tensor, idx: torch.Tensor, *,
                 scales: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 err_flag: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[r, j, :] = the cache row at position max(idx[r, j], 0) of row r's sequence, as bf16 [rows, n, d].

    idx: int32/int64 [rows, n], rows a multiple of the page table's b.  A position outside the page table or on
    a page outside the cache yields a zero row and sets ``err_flag``.
    """
    c = _cache_struct(cache, scales)
    dev = cache.device
    b, m, table_stride = _table(page_table, dev)
    rows, n, idx_stride = _index(idx, dev)
    d = c.d
    if out is not None and (out.shape != (rows, n, d) or not out.is_contiguous() or out.dtype != torch.bfloat16
                            or out.device != dev):
        raise ValueError("out must be a contiguous bf16 [rows, n, d] tensor")
    err = _flag(err_flag, dev)

    def call(s):
        to = torch.empty((rows, n, d), dtype=torch.bfloat16, device=dev) if out is None else out
        return _native.load().sel_cache_gather(
            c, page_table.data_ptr(), b, m, table_stride, idx.data_ptr(), _IDX[idx.dtype], rows, n, idx_stride,
            to.data_ptr(), err, s), to

    st, to = _launch(dev, stream, call)
    _native.check(st, "sel_cache_gather")
    return to


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
    gives zeros and a log-sum of -inf.  Positions a row does not attend to never influence it.  Should a wait inside
    the kernel run out (about 2 s), ``err_flag`` gets SEL_ETIMEOUT and the rows lost by it are NaN.

    Returns ``(out, lse)``: bf16 [rows, h, dv], and fp32 [rows, h] (natural log of the sum of exponentials) with
    ``return_lse``, else None.
    """
    c = _cache_struct(cache, scales)
    dev = cache.device
    b, m, table_stride = _table(page_table, dev)
    d = c.d
    if q.dtype != torch.bfloat16 or q.dim() != 3 or q.device != dev or q.shape[2] != d:
        raise ValueError("q must be a bfloat16 tensor [rows, h, d] on the cache's device")
    rows, h, _ = q.shape
    q_row, q_head, one = q.stride()
    if one != 1 and d > 1:
        raise ValueError("q must be contiguous in its last dimension")
    if end is not None and (end.dtype != torch.int32 or end.dim() != 1 or end.shape[0] != rows or end.device != dev
                            or not end.is_contiguous()):
        raise ValueError("end must be a contiguous int32 tensor with one entry per row")
    dv = d if dv is None else int(dv)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    n = idx_stride = idx_type = 0
    idx_ptr = None
    if idx is not None:
        listed, n, idx_stride = _index(idx, dev)
        if listed != rows:
            raise ValueError("idx must have one row per row of q")
        idx_type = _IDX[idx.dtype]
        # an empty list has no address of its own: any says that idx was given, and that of q has the alignment
        idx_ptr = idx.data_ptr() if n > 0 else q.data_ptr()
    if out is not None and (out.shape != (rows, h, dv) or not out.is_contiguous() or out.dtype != torch.bfloat16
                            or out.device != dev):
        raise ValueError("out must be a contiguous bf16 [rows, h, dv] tensor")
    err = _flag(err_flag, dev)

    def call(s):
        lib = _native.load()
        to = torch.empty((rows, h, max(dv, 0)), dtype=torch.bfloat16, device=dev) if out is None else out
        lse = torch.empty((rows, h), dtype=torch.float32, device=dev) if return_lse else None
        need = _scratch_bytes(dev.index, rows, h, d, dv, b, m, c.page_size, idx_ptr is not None, n)
        # Scratch of the call's own, from the stream's pool: two launches pass data through it, and another thread's
        # call on the same stream may come between them.
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        return lib.sel_cache_attention(
            q.data_ptr(), rows, h, q_row if rows > 1 else h * d, q_head if h > 1 else d, c, page_table.data_ptr(),
            b, m, table_stride, None if end is None else end.data_ptr(), idx_ptr, idx_type, n, idx_stride, dv,
            scale, to.data_ptr(), None if lse is None else lse.data_ptr(), None if ws is None else ws.data_ptr(),
            need, err, s), to, lse

    st, to, lse = _launch(dev, stream, call)
    _native.check(st, "sel_cache_attention")
    return to, lse
