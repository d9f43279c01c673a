"""Binding of the key/value cache and attention calls (include/qw3.h): argument
checks and marshalling only, like the package's other calls.

The cache of one layer is two tensors that the caller allocates (new_cache) and
keeps:
  codes  [pages, 2, H, page_size, D]  torch.int8 or torch.float8_e4m3fn
  scales [pages, 2, H, page_size]     float32
"""
from __future__ import annotations

import math

import torch

_CODE_TYPES = {torch.int8: 0, torch.float8_e4m3fn: 1}
_SRC_TYPES = {torch.bfloat16: 0, torch.float32: 1}
_BF16 = (torch.bfloat16,)

_lib = None
_fail = None


def _bind(lib, fail):
    """Called once by the package with the loaded library."""
    import ctypes
    global _lib, _fail
    _lib, _fail = lib, fail
    p, i, n, f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    lib.qcache_write.argtypes = [p, p, i, p, p, p, i] + [n] * 9 + [p]
    lib.qcache_read.argtypes = [p, p, i, p, p, p, p] + [n] * 7 + [p]
    lib.qattn_cache.argtypes = [p, p, p, i, p, p, p, p, p] + [n] * 10 + [f, p]
    lib.qattn_prompt.argtypes = [p] * 6 + [n] * 12 + [i, f, p]
    for name in ("qcache_write", "qcache_read", "qattn_cache", "qattn_prompt"):
        getattr(lib, name).restype = ctypes.c_int


# The stream as the C entry points take it. These calls take a few microseconds on
# the GPU, so what stands before a launch is kept short: the raw handle where
# torch offers it, one comparison for each property that is checked.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(index, fn, where, *args):
    if index == torch.cuda.current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        _fail(status, where)


def _rows(t, name, dtypes, index):
    """Checks of a [rows, heads, channels] operand: any strides, channels
    contiguous. Returns (token stride, head stride)."""
    if t.dtype not in dtypes:
        raise TypeError("%s must have dtype in %s, got %s" % (name, tuple(dtypes), t.dtype))
    if index < 0 or t.get_device() != index:
        raise ValueError("%s must be on the GPU device of the other arguments, got %s" % (name, t.device))
    if t.dim() != 3:
        raise ValueError("%s must be 3-D [rows, heads, channels], got shape %s" % (name, tuple(t.shape)))
    token, head, channel = t.stride()
    if channel != 1 and t.shape[2] > 1:
        raise ValueError("%s must be contiguous in its channels" % name)
    if (token | head) & 7:  # a dimension of one may have any stride; the others are the library's to check
        token, head = token if t.shape[0] > 1 else 0, head if t.shape[1] > 1 else 0
    return token, head


def _ints(t, name, dtype, index, shape):
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != index:
        raise ValueError("%s must be on GPU %d, got %s" % (name, index, t.device))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _cache(codes, scales):
    """(code type, device index, pages, H, page size, D) of a cache."""
    kind = _CODE_TYPES.get(codes.dtype)
    if kind is None:
        raise TypeError("codes must be int8 or float8_e4m3fn, got %s" % codes.dtype)
    shape = codes.shape
    if len(shape) != 5 or shape[1] != 2:
        raise ValueError("codes must be [pages, 2, H, page_size, D], got %s" % (tuple(shape),))
    if scales.dtype is not torch.float32 or scales.shape != shape[:4]:
        raise ValueError("scales must be float32 %s, got %s %s" % (tuple(shape[:4]), scales.dtype, tuple(scales.shape)))
    index = codes.get_device()
    if index < 0 or scales.get_device() != index:
        raise ValueError("codes and scales must be on one GPU device")
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError("codes and scales must be contiguous")
    pages, _, heads, size, dim = shape
    return kind, index, pages, heads, size, dim


def _table(block_table, index):
    if block_table.dim() != 2:
        raise ValueError("block_table must be [sequences, pages], got %s" % (tuple(block_table.shape),))
    _ints(block_table, "block_table", torch.int32, index, block_table.shape)
    return block_table.shape


def _scale(sm_scale, dim):
    return 1.0 / math.sqrt(dim) if sm_scale is None else sm_scale


def _out(out, like, shape):
    """`out` checked, or a new contiguous bf16 tensor of `shape` on like's device."""
    if out is None:
        if like.dtype is torch.bfloat16 and like.is_contiguous() and like.shape == shape:
            return torch.empty_like(like)
        return torch.empty(shape, dtype=torch.bfloat16, device=like.device)
    if out.dtype is not torch.bfloat16 or out.shape != shape or out.device != like.device or not out.is_contiguous():
        raise ValueError("out must be contiguous bfloat16 %s on %s" % (tuple(shape), like.device))
    return out


def new_cache(pages: int, page_size: int, heads: int, dim: int, dtype: torch.dtype = torch.int8, device="cuda"):
    """An empty cache (codes, scales) for qcache_write, qcache_read and qattn_cache."""
    if dtype not in _CODE_TYPES:
        raise TypeError("dtype must be int8 or float8_e4m3fn, got %s" % dtype)
    if dim not in (64, 128) or page_size < 16 or page_size > 65536 or page_size & (page_size - 1):
        raise ValueError("dim must be 64 or 128 and page_size a power of two in 16..65536")
    shape = (pages, 2, heads, page_size)
    return (torch.zeros(shape + (dim,), dtype=torch.uint8, device=device).view(dtype),
            torch.zeros(shape, dtype=torch.float32, device=device))


def qcache_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, codes: torch.Tensor,
                 scales: torch.Tensor) -> None:
    """Quantise k and v [T, H, D] (bf16 or float32) into the cache at slots
    [T] (int64, page * page_size + place, each at most once; negative: skip the token)."""
    kind, dev, pages, heads, size, dim = _cache(codes, scales)
    kts, khs = _rows(k, "k", _SRC_TYPES, dev)
    vts, vhs = _rows(v, "v", (k.dtype,), dev)
    shape = k.shape
    if v.shape != shape or shape[1] != heads or shape[2] != dim:
        raise ValueError("k and v must be [T, %d, %d], got %s and %s" % (heads, dim, tuple(shape), tuple(v.shape)))
    _ints(slots, "slots", torch.int64, dev, shape[:1])
    _call(dev, _lib.qcache_write, "qcache_write", k.data_ptr(), v.data_ptr(), _SRC_TYPES[k.dtype], slots.data_ptr(),
          codes.data_ptr(), scales.data_ptr(), kind, shape[0], heads, dim, pages, size, kts, khs, vts, vhs)


def qcache_read(codes: torch.Tensor, scales: torch.Tensor, block_table: torch.Tensor, cu: torch.Tensor, total: int,
                out=None):
    """The sequences' cached tokens as dense bf16 (k, v), each [total, H, D]:
    row cu[b] + n is token n of sequence b."""
    kind, dev, pages, heads, size, dim = _cache(codes, scales)
    batch, max_pages = _table(block_table, dev)
    _ints(cu, "cu", torch.int32, dev, (batch + 1,))
    if total < 0:
        raise ValueError("total must not be negative")
    if out is None:
        k, v = torch.empty((2, total, heads, dim), dtype=torch.bfloat16, device=codes.device).unbind(0)
    else:
        k, v = (_out(t, codes, (total, heads, dim)) for t in out)
    _call(dev, _lib.qcache_read, "qcache_read", codes.data_ptr(), scales.data_ptr(), kind, block_table.data_ptr(),
          cu.data_ptr(), k.data_ptr(), v.data_ptr(), batch, max_pages, total, heads, dim, pages, size)
    return k, v


def qattn_cache(q: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, block_table: torch.Tensor,
                lens: torch.Tensor, cu_q: torch.Tensor | None = None, tree: torch.Tensor | None = None,
                sm_scale: float | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of new tokens q [Tq, Hq, D] (bf16) over the quantised cache.

    lens [B] counts each sequence's cached tokens, its new ones included (they
    are its last). cu_q [B + 1]: the new tokens of each sequence (None: one
    each). tree [Tq] int64: bit j of a row's word lets it see new token j < 64
    of its sequence (None: causal). sm_scale defaults to 1/sqrt(D)."""
    kind, dev, pages, heads, size, dim = _cache(codes, scales)
    qts, qhs = _rows(q, "q", _BF16, dev)
    rows, hq, d = shape = q.shape
    if d != dim or hq % heads:
        raise ValueError("q must be [rows, a multiple of %d, %d], got %s" % (heads, dim, tuple(shape)))
    batch, max_pages = _table(block_table, dev)
    _ints(lens, "lens", torch.int32, dev, (batch,))
    if cu_q is not None:
        _ints(cu_q, "cu_q", torch.int32, dev, (batch + 1,))
    elif rows != batch:
        raise ValueError("without cu_q, q must have one row for each of the %d sequences, got %d" % (batch, rows))
    if tree is not None:
        _ints(tree, "tree", torch.int64, dev, (rows,))
    out = _out(out, q, shape)
    _call(dev, _lib.qattn_cache, "qattn_cache", q.data_ptr(), codes.data_ptr(), scales.data_ptr(), kind,
          block_table.data_ptr(), lens.data_ptr(), cu_q.data_ptr() if cu_q is not None else None,
          tree.data_ptr() if tree is not None else None, out.data_ptr(), batch, max_pages, rows, hq, heads, dim, pages,
          size, qts, qhs, _scale(sm_scale, dim))
    return out


def qattn_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                 cu_k: torch.Tensor | None = None, causal: bool = True, sm_scale: float | None = None,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of packed prompts: q [Tq, Hq, D] over k, v [Tk, H, D] (bf16),
    sequence b owning rows cu_q[b] .. cu_q[b + 1] - 1 and keys cu_k likewise
    (None: cu_q). Causal rows are aligned at the end: row i of nq sees the keys
    j <= i + nk - nq. sm_scale defaults to 1/sqrt(D)."""
    dev = q.get_device()
    qts, qhs = _rows(q, "q", _BF16, dev)
    kts, khs = _rows(k, "k", _BF16, dev)
    vts, vhs = _rows(v, "v", _BF16, dev)
    rows, hq, dim = shape = q.shape
    keys, heads, d = k.shape
    if v.shape != k.shape or d != dim or heads == 0 or hq % heads:
        raise ValueError("k and v must be [keys, a divisor of %d, %d], got %s and %s"
                         % (hq, dim, tuple(k.shape), tuple(v.shape)))
    if dim not in (64, 128):
        raise ValueError("channels must be 64 or 128, got %d" % dim)
    if cu_q.dim() != 1 or cu_q.shape[0] < 1:
        raise ValueError("cu_q must be [sequences + 1], got %s" % (tuple(cu_q.shape),))
    _ints(cu_q, "cu_q", torch.int32, dev, cu_q.shape)
    if cu_k is None:
        cu_k = cu_q
    else:
        _ints(cu_k, "cu_k", torch.int32, dev, cu_q.shape)
    out = _out(out, q, shape)
    _call(dev, _lib.qattn_prompt, "qattn_prompt", q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_q.data_ptr(),
          cu_k.data_ptr(), out.data_ptr(), cu_q.shape[0] - 1, rows, keys, hq, heads, dim, qts, qhs, kts, khs, vts, vhs,
          1 if causal else 0, _scale(sm_scale, dim))
    return out
