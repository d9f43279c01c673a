"""Binding of the rotary position calls (include/qw3.h): argument checks and
marshalling only, like the package's other calls."""
from __future__ import annotations

import torch

from ._attention import _BF16, _SRC_TYPES, _cache, _call, _ints, _out, _rows

_STYLES = {"halves": 0, "pairs": 1}

_lib = None


def _bind(lib):
    """Called once by the package with the loaded library."""
    import ctypes
    global _lib
    _lib = lib
    p, i, n = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.qrope.argtypes = [p, i, p, p, p, i, p] + [n] * 7 + [p]
    lib.qrope_write.argtypes = [p, p, p, i, p, p, p, i, p, p, p, p, p, p, i] + [n] * 14 + [p]
    for name in ("qrope", "qrope_write"):
        getattr(lib, name).restype = ctypes.c_int


def _angles(positions, rates, axis, style, tokens, index):
    """(style, axes, rotated channels) of a rotation."""
    kind = _STYLES.get(style)
    if kind is None:
        raise ValueError('style must be "halves" or "pairs", got %r' % (style,))
    shape, pairs = positions.shape, rates.shape
    axes = shape[0] if len(shape) == 2 else 1
    _ints(positions, "positions", torch.int32, index, (axes, tokens) if len(shape) == 2 else (tokens,))
    if len(pairs) != 1:
        raise ValueError("rates must be [pairs], got %s" % (tuple(pairs),))
    _ints(rates, "rates", torch.float64, index, pairs)
    if axis is not None:
        _ints(axis, "axis", torch.int32, index, pairs)
    return kind, axes, 2 * pairs[0]


def qrope(x: torch.Tensor, positions: torch.Tensor, rates: torch.Tensor, axis: torch.Tensor | None = None,
          style: str = "halves", out: torch.Tensor | None = None) -> torch.Tensor:
    """Rows x [T, H, D] (bf16 or float32) with their first 2 * len(rates)
    channels rotated; bf16 [T, H, D].

    positions int32 [T], or [A, T] for A axes; rates float64 [pairs], radians
    for each position; axis int32 [pairs]: the axis of each pair (None: axis 0).
    style: a pair is the channels (i, i + pairs) ("halves") or (2 i, 2 i + 1) ("pairs")."""
    dev = x.get_device()
    xts, xhs = _rows(x, "x", _SRC_TYPES, dev)
    tokens, heads, dim = shape = x.shape
    kind, axes, rotated = _angles(positions, rates, axis, style, tokens, dev)
    out = _out(out, x, shape)
    _call(dev, _lib.qrope, "qrope", x.data_ptr(), _SRC_TYPES[x.dtype], positions.data_ptr(), rates.data_ptr(),
          axis.data_ptr() if axis is not None else None, kind, out.data_ptr(), tokens, heads, dim, rotated, axes, xts, xhs)
    return out


def qrope_write(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, rates: torch.Tensor,
                slots: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, axis: torch.Tensor | None = None,
                style: str = "halves", dense: bool = False, out=None):
    """Rotate q [T, Hq, D] and k [T, H, D] as qrope does, and store k and v
    [T, H, D] in the cache as qcache_write does, in one pass.

    Returns the rotated q (bf16), or with `dense` (q, k, v), all bf16 and
    contiguous, for qattn_prompt. q, k and v have one dtype, bf16 or float32.
    `out`: what is returned, allocated by the caller."""
    kind, dev, pages, heads, size, dim = _cache(codes, scales)
    qts, qhs = _rows(q, "q", _SRC_TYPES, dev)
    kts, khs = _rows(k, "k", (q.dtype,), dev)
    vts, vhs = _rows(v, "v", (q.dtype,), dev)
    tokens, hq, d = q.shape
    shape = k.shape
    if d != dim or hq % heads or v.shape != shape or shape != (tokens, heads, dim):
        raise ValueError("q must be [T, a multiple of %d, %d], k and v [T, %d, %d], got %s, %s and %s"
                         % (heads, dim, heads, dim, tuple(q.shape), tuple(k.shape), tuple(v.shape)))
    _ints(slots, "slots", torch.int64, dev, (tokens,))
    how, axes, rotated = _angles(positions, rates, axis, style, tokens, dev)
    if dense:
        qo, ko, vo = (_out(t, like, like.shape) for t, like in zip(out if out is not None else (None,) * 3, (q, k, v)))
    else:
        qo, ko, vo = _out(out, q, q.shape), None, None
    _call(dev, _lib.qrope_write, "qrope_write", q.data_ptr(), k.data_ptr(), v.data_ptr(), _SRC_TYPES[q.dtype],
          positions.data_ptr(), rates.data_ptr(), axis.data_ptr() if axis is not None else None, how, slots.data_ptr(),
          qo.data_ptr(), ko.data_ptr() if dense else None, vo.data_ptr() if dense else None, codes.data_ptr(),
          scales.data_ptr(), kind, tokens, hq, heads, dim, rotated, axes, pages, size, qts, qhs, kts, khs, vts, vhs)
    return (qo, ko, vo) if dense else qo
