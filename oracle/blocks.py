"""Attention over selected pages of the cache, page by page and row by row, from
the definitions (include/qw3.h).  Shares no code with the GPU path.

Bounds and scores are whole numbers and single float32 operations by definition,
so they are computed in those; attention is in 64 bits (oracle/attention.py)."""
import numpy as np

from oracle import attention as ref
from oracle.pages import starts_of


def rows_of(lens, cu, total, room):
    """(row, sequence, position) of each row that belongs to a sequence."""
    got = []
    for b, (first, n) in enumerate(starts_of(cu, len(lens), total)):
        length = min(max(int(lens[b]), 0), room)
        got += [(first + i, b, length - n + i) for i in range(n)]
    return got


def codes_of(y):
    """float32 numbers under one scale, max / 127: (int8 numbers, scale); what is not finite: zeros and NaN."""
    y = np.asarray(y, np.float32)
    if not np.isfinite(y).all():
        return np.zeros(y.shape, np.int8), np.float32(np.nan)
    s = np.float32(np.abs(y).max() / np.float32(127))
    if not s > 0:
        return np.zeros(y.shape, np.int8), s
    return np.rint(np.clip((y / s).astype(np.float32), -127, 127)).astype(np.int8), s


def bounds(codes, scales, kind, table, lens, cu, total, size, out, out_scales):
    """out [pages, H, 2, D] int8 and out_scales [pages, H] are updated."""
    width, pages = table.shape[1], codes.shape[0]
    for b, (_, n) in enumerate(starts_of(cu, len(lens), total)):
        length = min(max(int(lens[b]), 0), width * size)
        if n == 0:
            continue
        for c in range(max(length - n, 0) // size, -(-length // size)):
            page = table[b, c]
            if not 0 <= page < pages:
                continue
            used = min(size, length - c * size)
            with np.errstate(all="ignore"):
                x = ref.code_values(codes[page, 0, :, :used], kind).astype(np.float32) * scales[page, 0, :, :used, None]
            for h in range(codes.shape[2]):
                ends = np.stack([x[h].max(0), x[h].min(0)]) if np.isfinite(x[h]).all() and np.isfinite(scales[page, 0, h, :used]).all() \
                    else np.full((2, x.shape[2]), np.nan)
                out[page, h], out_scales[page, h] = codes_of(ends)


def sums_of(mine):
    """A kv head's queries [queries, D] float64: the sums of their positive and negative values [2, D], in 64 bits and in
    their order, as float32 numbers; where one passes those, all times 2^-16."""
    sums = np.zeros((2, mine.shape[1]))
    for x in mine:
        sums[0] += np.maximum(x, 0)
        sums[1] += np.minimum(x, 0)
    with np.errstate(over="ignore"):
        single = sums.astype(np.float32)
    return (sums * 2.0 ** -16).astype(np.float32) if np.isfinite(sums).all() and not np.isfinite(single).all() else single


def select(q, limits, steps, table, lens, cu, count, size, first, recent):
    """picks [rows, H, count]; q [rows, Hq, D] in float64, limits int8 [pages, H, 2, D], steps float32 [pages, H]. Rows of
    no sequence: -9."""
    rows, hq, dim = q.shape
    pages, heads = steps.shape
    picks = np.full((rows, heads, count), -9, np.int32)
    for t, b, pos in rows_of(lens, cu, rows, table.shape[1] * size):
        seen = 0 if pos < 0 else pos // size + 1
        for h in range(heads):
            picks[t, h] = -1
            if seen <= count:
                picks[t, h, :seen] = np.arange(seen)
                continue
            mine = q[t, h * (hq // heads):(h + 1) * (hq // heads)]
            w = codes_of(sums_of(mine))[0].astype(np.int64)
            page = table[b, :seen]
            there = (page >= 0) & (page < pages)
            at = np.where(there, page, 0)
            sums = (limits[at, h].astype(np.int64) * w).sum((1, 2))
            with np.errstate(all="ignore"):
                score = sums.astype(np.float32) * steps[at, h]
            # NaN first, then by size, pages that are not there last; of equals the lower place
            rank = np.where(np.isnan(score), 2, 1) * there
            order = [i for i in sorted(range(first, seen - recent), key=lambda i: (-rank[i], -score[i] if rank[i] == 1 else 0, i))]
            taken = list(range(first)) + order[:count - first - recent] + list(range(seen - recent, seen))
            picks[t, h] = sorted(taken)
    return picks


def tokens_of(picks, size, pos, page, pages):
    """The positions, with repetition, that a row at `pos` sees through its picks, as many of them as it sees pages; page: its
    sequence's row of the table."""
    got = []
    for p in picks[:0 if pos < 0 else pos // size + 1]:
        if 0 <= p < len(page) and 0 <= page[p] < pages:
            got += [t for t in range(p * size, (p + 1) * size) if t <= pos]
    return np.array(got, int)
