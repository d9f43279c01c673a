"""Binding of the calls on the cache's pages (include/qw3.h): argument checks and
marshalling only, like the package's other calls.

Who holds a page is counted in a tensor that the caller allocates with the cache
and keeps: refs [pages] int32, zeros at first.  A block table starts as -1 in
every entry, lengths as 0.  page_size is the cache's, which qcache_reserve and
qcache_fork do not see and cannot check.  A cache of several layers is codes [layers, pages, 2,
H, page_size, D] and scales [layers, pages, 2, H, page_size]; codes[i] and
scales[i] are what the calls of one layer take.
"""
from __future__ import annotations

import torch

from ._attention import _CODE_TYPES, _call, _ints, _table

_lib = None


def _bind(lib):
    """Called once by the package with the loaded library."""
    import ctypes
    global _lib
    _lib = lib
    p, n = ctypes.c_void_p, ctypes.c_int64
    lib.qcache_reserve.argtypes = [p] * 7 + [n] * 5 + [p]
    lib.qcache_fork.argtypes = [p] * 6 + [n] * 5 + [p]
    lib.qcache_copy.argtypes = [p] * 3 + [n] * 6 + [p]
    lib.qcache_compact.argtypes = [p] * 7 + [n] * 8 + [p]
    for name in ("qcache_reserve", "qcache_fork", "qcache_copy", "qcache_compact"):
        getattr(lib, name).restype = ctypes.c_int


def _layers(codes, scales):
    """(device index, layers, pages, H, page size, D) of a cache of one layer or several."""
    if codes.dtype not in _CODE_TYPES:
        raise TypeError("codes must be int8 or float8_e4m3fn, got %s" % codes.dtype)
    shape = codes.shape
    if len(shape) not in (5, 6) or shape[-4] != 2:
        raise ValueError("codes must be [pages, 2, H, page_size, D], or that with the layers in front, got %s" % (tuple(shape),))
    if scales.dtype is not torch.float32 or scales.shape != shape[:-1]:
        raise ValueError("scales must be float32 %s, got %s %s" % (tuple(shape[:-1]), scales.dtype, tuple(scales.shape)))
    index = codes.get_device()
    if index < 0 or scales.get_device() != index:
        raise ValueError("codes and scales must be on one GPU device")
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError("codes and scales must be contiguous")
    return index, shape[0] if len(shape) == 6 else 1, shape[-5], shape[-3], shape[-2], shape[-1]


def _held(refs, block_table, lens):
    """(device index, pages, sequences, entries of a sequence)."""
    index = refs.get_device()
    if index < 0 or refs.dim() != 1:
        raise ValueError("refs must be [pages] on a GPU device, got %s on %s" % (tuple(refs.shape), refs.device))
    _ints(refs, "refs", torch.int32, index, refs.shape)
    batch, max_pages = _table(block_table, index)
    _ints(lens, "lens", torch.int32, index, (batch,))
    return index, refs.shape[0], batch, max_pages


def qcache_reserve(refs: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor, page_size: int,
                   cu: torch.Tensor | None = None, total: int | None = None):
    """Room for new tokens behind each sequence's last: (slots, lens, copies).

    cu [B + 1] int32 and total: the new tokens of each sequence and of all
    (None: one each). refs and block_table are updated. slots [total] int64 are
    what qcache_write and qrope_write take, -1 where there was no room; lens [B]
    the new lengths; copies [B, 2] what qcache_copy has to copy first."""
    dev, pages, batch, max_pages = _held(refs, block_table, lens)
    if cu is None:
        if total is not None and total != batch:
            raise ValueError("without cu there is one new token for each of the %d sequences, got total %d" % (batch, total))
        total = batch
    else:
        _ints(cu, "cu", torch.int32, dev, (batch + 1,))
        if total is None or total < 0:
            raise ValueError("with cu, total must say how many new tokens there are")
    slots = lens.new_empty((total,), dtype=torch.int64)
    lens_out = torch.empty_like(lens)
    copies = lens.new_empty((batch, 2))
    _call(dev, _lib.qcache_reserve, "qcache_reserve", refs.data_ptr(), block_table.data_ptr(), lens.data_ptr(),
          cu.data_ptr() if cu is not None else None, slots.data_ptr(), lens_out.data_ptr(), copies.data_ptr(), batch,
          max_pages, total, pages, page_size)
    return slots, lens_out, copies


def qcache_fork(refs: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor, parents: torch.Tensor, page_size: int):
    """(block table, lens) in which sequence b follows sequence parents[b] (int32,
    any number of them; a parent that is no sequence: an empty one). refs is
    updated: the new table's entries hold the pages, the old one's no longer do."""
    dev, pages, batch, max_pages = _held(refs, block_table, lens)
    if parents.dim() != 1:
        raise ValueError("parents must be [sequences], got %s" % (tuple(parents.shape),))
    _ints(parents, "parents", torch.int32, dev, parents.shape)
    count = parents.shape[0]
    table_out = torch.empty_like(block_table) if count == batch else lens.new_empty((count, max_pages))
    lens_out = torch.empty_like(parents)
    _call(dev, _lib.qcache_fork, "qcache_fork", refs.data_ptr(), block_table.data_ptr(), lens.data_ptr(), parents.data_ptr(),
          table_out.data_ptr(), lens_out.data_ptr(), batch, count, max_pages, pages, page_size)
    return table_out, lens_out


def qcache_copy(codes: torch.Tensor, scales: torch.Tensor, copies: torch.Tensor) -> None:
    """Copy the pages copies [n, 2] (int32: from, to; negative: none), in every
    layer of the cache. A page that is written is neither read nor written by another pair."""
    dev, layers, pages, heads, size, dim = _layers(codes, scales)
    if copies.dim() != 2:
        raise ValueError("copies must be [n, 2], got %s" % (tuple(copies.shape),))
    _ints(copies, "copies", torch.int32, dev, (copies.shape[0], 2))
    _call(dev, _lib.qcache_copy, "qcache_copy", codes.data_ptr(), scales.data_ptr(), copies.data_ptr(), copies.shape[0],
          layers, heads, dim, pages, size)


def qcache_compact(codes: torch.Tensor, scales: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor,
                   keep: torch.Tensor, cu_q: torch.Tensor | None = None) -> torch.Tensor:
    """Drop, in place and in every layer, those of each sequence's last tokens that
    keep (bool or uint8 [Tq], cu_q [B + 1] as in qattn_cache; None: one each) does
    not keep; the others move up in order. Returns the new lengths."""
    dev, layers, pages, heads, size, dim = _layers(codes, scales)
    batch, max_pages = _table(block_table, dev)
    _ints(lens, "lens", torch.int32, dev, (batch,))
    if keep.dim() != 1:
        raise ValueError("keep must be [tokens], got %s" % (tuple(keep.shape),))
    _ints(keep, "keep", torch.bool if keep.dtype is torch.bool else torch.uint8, dev, keep.shape)
    if cu_q is not None:
        _ints(cu_q, "cu_q", torch.int32, dev, (batch + 1,))
    elif keep.shape[0] != batch:
        raise ValueError("without cu_q, keep must have one entry for each of the %d sequences, got %d" % (batch, keep.shape[0]))
    lens_out = torch.empty_like(lens)
    _call(dev, _lib.qcache_compact, "qcache_compact", codes.data_ptr(), scales.data_ptr(), block_table.data_ptr(),
          lens.data_ptr(), cu_q.data_ptr() if cu_q is not None else None, keep.data_ptr(), lens_out.data_ptr(), batch,
          max_pages, keep.shape[0], layers, heads, dim, pages, size)
    return lens_out
