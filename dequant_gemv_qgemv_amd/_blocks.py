"""Binding of the calls that attend over some of the cache's pages
(include/qw3.h): argument checks and marshalling only, like the package's other
calls.

Beside the cache of a layer the caller keeps the bounds of its pages' keys
(new_bounds):
  bounds        [pages, H, 2, D]  int8
  bound_scales  [pages, H]        float32
"""
from __future__ import annotations

import torch

from ._attention import _BF16, _cache, _call, _ints, _out, _rows, _scale, _table

_lib = None


def _bind(lib):
    """Called once by the package with the loaded library."""
    import ctypes
    global _lib
    _lib = lib
    p, i, n, f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    lib.qcache_bounds.argtypes = [p, p, i, p, p, p, p, p] + [n] * 7 + [p]
    lib.qblock_select.argtypes = [p] * 7 + [n] * 13 + [p]
    lib.qattn_blocks.argtypes = [p, p, p, i, p, p, p, p, p] + [n] * 11 + [f, p]
    for name in ("qcache_bounds", "qblock_select", "qattn_blocks"):
        getattr(lib, name).restype = ctypes.c_int


def new_bounds(codes: torch.Tensor):
    """Bounds (bounds, bound_scales) beside a layer's cache codes, for qcache_bounds and qblock_select."""
    pages, _, heads, _, dim = codes.shape
    return (torch.zeros((pages, heads, 2, dim), dtype=torch.int8, device=codes.device),
            torch.zeros((pages, heads), dtype=torch.float32, device=codes.device))


def _bounds(bounds, bound_scales, index):
    """(pages, H, D) of bounds."""
    shape = bounds.shape
    if bounds.dtype is not torch.int8:
        raise TypeError("bounds must be int8, got %s" % bounds.dtype)
    if len(shape) != 4 or shape[2] != 2:
        raise ValueError("bounds must be [pages, H, 2, D], got %s" % (tuple(shape),))
    if bound_scales.dtype is not torch.float32 or bound_scales.shape != shape[:2]:
        raise ValueError("bound_scales must be float32 %s, got %s %s" % (tuple(shape[:2]), bound_scales.dtype, tuple(bound_scales.shape)))
    if bounds.get_device() != index or bound_scales.get_device() != index:
        raise ValueError("bounds and bound_scales must be on GPU %d" % index)
    if not (bounds.is_contiguous() and bound_scales.is_contiguous()):
        raise ValueError("bounds and bound_scales must be contiguous")
    return shape[0], shape[1], shape[3]


def _sequences(block_table, lens, cu_q, rows, index):
    """(sequences, entries of the table) of a call with `rows` new tokens."""
    batch, max_pages = _table(block_table, index)
    _ints(lens, "lens", torch.int32, index, (batch,))
    if cu_q is not None:
        _ints(cu_q, "cu_q", torch.int32, index, (batch + 1,))
    elif rows != batch:
        raise ValueError("without cu_q there must be one row for each of the %d sequences, got %d" % (batch, rows))
    return batch, max_pages


def qcache_bounds(codes: torch.Tensor, scales: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor,
                  bounds: torch.Tensor, bound_scales: torch.Tensor, cu_q: torch.Tensor | None = None,
                  total: int | None = None) -> None:
    """The bounds of the pages that hold the sequences' new tokens, once those are
    in the cache: their last tokens, counted by cu_q [B + 1] and, all together, total (None: one each)."""
    kind, dev, pages, heads, size, dim = _cache(codes, scales)
    if _bounds(bounds, bound_scales, dev) != (pages, heads, dim):
        raise ValueError("bounds must be [%d, %d, 2, %d], got %s" % (pages, heads, dim, tuple(bounds.shape)))
    if total is None:
        if cu_q is not None:
            raise ValueError("with cu_q, total must say how many new tokens there are")
        total = lens.shape[0] if lens.dim() == 1 else 0
    if total < 0:
        raise ValueError("total must not be negative")
    batch, max_pages = _sequences(block_table, lens, cu_q, total, dev)
    _call(dev, _lib.qcache_bounds, "qcache_bounds", codes.data_ptr(), scales.data_ptr(), kind, block_table.data_ptr(),
          lens.data_ptr(), cu_q.data_ptr() if cu_q is not None else None, bounds.data_ptr(), bound_scales.data_ptr(), batch,
          max_pages, total, heads, dim, pages, size)


def qblock_select(q: torch.Tensor, bounds: torch.Tensor, bound_scales: torch.Tensor, block_table: torch.Tensor,
                  lens: torch.Tensor, count: int, page_size: int, cu_q: torch.Tensor | None = None, first: int = 1,
                  recent: int = 1, out: torch.Tensor | None = None) -> torch.Tensor:
    """The pages that rows q [Tq, Hq, D] (bf16; new tokens as in qattn_cache) attend
    to: int32 [Tq, H, count] places in their sequence's block table, ascending, -1 behind the last.

    All where a row sees at most count; else its first ones, its recent ones
    (its own is the last) and those with the highest scores by the bounds.
    page_size is the cache's, which this call does not see and cannot check."""
    dev = q.get_device()
    qts, qhs = _rows(q, "q", _BF16, dev)
    pages, heads, dim = _bounds(bounds, bound_scales, dev)
    rows, hq, d = q.shape
    if d != dim or heads == 0 or hq % heads:
        raise ValueError("q must be [rows, a multiple of %d, %d], got %s" % (heads, dim, tuple(q.shape)))
    batch, max_pages = _sequences(block_table, lens, cu_q, rows, dev)
    if count < 1 or first < 0 or recent < 1 or first + recent > count:
        raise ValueError("count must be at least first + recent, first at least 0 and recent at least 1, got %d, %d, %d"
                         % (count, first, recent))
    shape = (rows, heads, count)
    if out is None:
        out = lens.new_empty(shape)
    else:
        _ints(out, "out", torch.int32, dev, shape)
    _call(dev, _lib.qblock_select, "qblock_select", q.data_ptr(), bounds.data_ptr(), bound_scales.data_ptr(),
          block_table.data_ptr(), lens.data_ptr(), cu_q.data_ptr() if cu_q is not None else None, out.data_ptr(), batch,
          max_pages, rows, hq, heads, dim, pages, page_size, count, first, recent, qts, qhs)
    return out


def qattn_blocks(q: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, block_table: torch.Tensor,
                 lens: torch.Tensor, picks: torch.Tensor, cu_q: torch.Tensor | None = None, sm_scale: float | None = None,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of new tokens q [Tq, Hq, D] (bf16) over the tokens, up to their own,
    of the pages picks [Tq, H, count]: places in their sequence's block table in
    any order, of which as many are read as the row sees pages (others than 0 ..
    the table's width - 1: none). Sequences as in qattn_cache."""
    kind, dev, pages, heads, size, dim = _cache(codes, scales)
    qts, qhs = _rows(q, "q", _BF16, dev)
    rows, hq, d = shape = q.shape
    if d != dim or hq % heads:
        raise ValueError("q must be [rows, a multiple of %d, %d], got %s" % (heads, dim, tuple(shape)))
    batch, max_pages = _sequences(block_table, lens, cu_q, rows, dev)
    if picks.dim() != 3:
        raise ValueError("picks must be [rows, %d, count], got %s" % (heads, tuple(picks.shape)))
    count = picks.shape[2]
    _ints(picks, "picks", torch.int32, dev, (rows, heads, count))
    out = _out(out, q, shape)
    _call(dev, _lib.qattn_blocks, "qattn_blocks", q.data_ptr(), codes.data_ptr(), scales.data_ptr(), kind,
          block_table.data_ptr(), lens.data_ptr(), cu_q.data_ptr() if cu_q is not None else None, picks.data_ptr(),
          out.data_ptr(), batch, max_pages, rows, hq, heads, dim, pages, size, count, qts, qhs, _scale(sm_scale, dim))
    return out
