"""The pages of the key/value cache, one sequence, entry and token after the
other, from their definitions (include/qw3.h).  Shares no code with the GPU path."""
import numpy as np


def starts_of(cu, batch, total):
    """First row and number of rows of each sequence: a start below an earlier one counts as that one."""
    if cu is None:
        return [(b, 1) for b in range(batch)]
    got, floor = [], 0
    for b in range(batch):
        first = max(min(max(int(cu[b]), 0), total), floor)
        got.append((first, max(min(max(int(cu[b + 1]), 0), total) - first, 0)))
        floor = first
    return got


def reserve(refs, table, lens, cu, total, size):
    """(slots, lens, copies); refs and table are updated."""
    batch, width = table.shape
    pages = len(refs)
    free = [p for p in range(pages) if refs[p] == 0]
    before = refs.copy()
    slots = np.full(total, -1, np.int64)
    lens_out = np.zeros(batch, np.int32)
    copies = np.full((batch, 2), -1, np.int32)
    closed = False  # once a sequence's needs were not met
    for b, (first, n) in enumerate(starts_of(cu, batch, total)):
        length = min(max(int(lens[b]), 0), width * size)
        lens_out[b] = length
        if length + n > width * size or n == 0:
            continue
        reach = range(length // size, -(-(length + n) // size))
        needs = [c for c in reach if not 0 <= table[b, c] < pages or before[table[b, c]] > 1]
        if needs and (closed or len(needs) > len(free)):
            closed = True
            continue
        for c in needs:
            page, old = free.pop(0), table[b, c]
            if 0 <= old < pages:
                refs[old] -= 1
                if c == length // size and length % size:
                    copies[b] = old, page
            table[b, c] = page
            refs[page] = 1
        lens_out[b] = length + n
        for i in range(n):
            slots[first + i] = int(table[b, (length + i) // size]) * size + (length + i) % size
    return slots, lens_out, copies


def fork(refs, table, lens, parents, size):
    """(table, lens); refs is updated."""
    batch, width = table.shape
    out, lens_out = np.full((len(parents), width), -1, np.int32), np.zeros(len(parents), np.int32)
    for p in table.reshape(-1):
        if 0 <= p < len(refs):
            refs[p] -= 1
    for b, parent in enumerate(parents):
        if not 0 <= parent < batch:
            continue
        lens_out[b] = min(max(int(lens[parent]), 0), width * size)
        for c in range(-(-int(lens_out[b]) // size)):
            if 0 <= table[parent, c] < len(refs):
                out[b, c] = table[parent, c]
                refs[out[b, c]] += 1
    return out, lens_out


def copy(codes, scales, copies):
    """codes [layers, pages, ...] and scales are updated."""
    for a, b in copies:
        if 0 <= a < codes.shape[1] and 0 <= b < codes.shape[1]:
            codes[:, b], scales[:, b] = codes[:, a], scales[:, a]


def compact(codes, scales, table, lens, keep, cu, size):
    """New lengths; codes [layers, pages, 2, H, size, D] and scales are updated."""
    batch, width = table.shape
    pages = codes.shape[1]
    lens_out = np.zeros(batch, np.int32)
    for b, (first, n) in enumerate(starts_of(cu, batch, len(keep))):
        length = min(max(int(lens[b]), 0), width * size)
        to = max(length - n, 0)
        for i in range(n):
            at = length - n + i
            if at < 0 or not keep[first + i]:
                continue
            src, dst = table[b, at // size], table[b, to // size]
            if 0 <= dst < pages:
                there = 0 <= src < pages
                codes[:, dst, :, :, to % size] = codes[:, src, :, :, at % size] if there else 0
                scales[:, dst, :, :, to % size] = scales[:, src, :, :, at % size] if there else 0
            to += 1
        lens_out[b] = to
    return lens_out
