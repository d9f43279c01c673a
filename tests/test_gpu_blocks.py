"""Attention over selected pages on the GPU: bounds and selections equal to
oracle/blocks.py's in every number, outputs inside the bound that
oracle/attention.py derives for each (attend)."""
import math
import sys

import numpy as np
import pytest
import torch

from oracle import attention as ref
from oracle import blocks

pytestmark = pytest.mark.gpu

TORCH = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def q():
    import dequant_gemv_qgemv_amd as mod
    return mod


def say(*args):
    print("[gpu-case]", *args, file=sys.stderr, flush=True)


def dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def rows(rng, n, heads, dim):
    return torch.tensor(rng.standard_normal((n, heads, dim)) * np.exp(rng.standard_normal((1, heads, dim))), dtype=torch.float32).to(torch.bfloat16).cuda()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def tables(rng, lens, size, spare=3, width=None, lost=0.0):
    """(block table, pages): pages in random order, some entries naming none."""
    need = [-(-max(int(n), 0) // size) for n in lens]
    pages = sum(need) + spare
    ids = rng.permutation(pages)
    table = np.full((len(lens), width or max(need) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    gone = rng.random(table.shape) < lost
    table[gone] = rng.choice([-1, pages, 1 << 30], gone.sum())
    return table, pages


def cache(rng, kind, pages, heads, size, dim):
    raw = rng.integers(0, 256, (pages, 2, heads, size, dim), dtype=np.uint8)
    if kind == "e4m3":
        raw[(raw & 0x7F) == 0x7F] = 0x3C  # no NaN unless a test puts it there
    scales = (rng.uniform(0.5, 2.0, (pages, 2, heads, size)) / (70 if kind == "int8" else 100)).astype(np.float32)
    return raw, scales


def on_gpu(raw, scales, kind):
    return torch.tensor(raw).cuda().view(TORCH[kind]), torch.tensor(scales).cuda()


# ----------------------------------------------------------------- bounds ---
BOUNDS = [  # page size, heads, channels, lengths, new tokens (None: one each)
    (16, 1, 64, [1], None), (16, 3, 128, [5, 16, 17, 200], None), (64, 8, 128, [1, 64, 65, 300], [1, 64, 2, 130]),
    (32, 2, 64, [500, 31, 0, 90], [500, 31, 0, 1]), (16, 5, 128, [700, 3], [33, 3]), (256, 2, 64, [255, 700], [255, 300]),
    (16, 2, 128, list(range(1, 90)), None), (128, 1, 128, [1000, 129, 128], [999, 129, 128])]


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("case", BOUNDS, ids=str)
def test_bounds(kind, case):
    say("bounds", kind, case)
    size, heads, dim, lens, new = case
    rng = np.random.default_rng(sum(lens) + size)
    table, pages = tables(rng, lens, size, lost=0.05 if len(lens) > 2 else 0.0)
    raw, scales = cache(rng, kind, pages, heads, size, dim)
    scales[rng.random(scales.shape) < 0.02] = 0.0
    page = table[-1, 0]
    if 0 <= page < pages and len(lens) > 1:
        scales[page, 0, 0] = 0.0                     # a page of zeros
        if heads > 1:
            scales[page, 0, 1] *= np.float32(1e-38)  # denormal scales
    if len(lens) > 3:  # what is not a number, in and behind the tokens there are
        for b, at, bad in ((1, 0, np.nan), (3, lens[3] - 1, np.inf)):
            p = table[b, at // size]
            if 0 <= p < pages:
                scales[p, 0, heads - 1, at % size] = bad
        p = table[0, (lens[0] - 1) // size]
        if 0 <= p < pages and lens[0] % size:
            scales[p, 0, :, lens[0] % size:] = np.nan
            raw[p, 0, :, lens[0] % size:] = 0xFF
        p = table[2, 0]
        if kind == "e4m3" and 0 <= p < pages:
            raw[p, 0, 0, 0, 3] = 0x7F
    cu = None if new is None else np.r_[0, np.cumsum(new)]
    total = len(lens) if new is None else int(cu[-1])
    want, want_s = np.full((pages, heads, 2, dim), 77, np.int8), np.full((pages, heads), -5.0, np.float32)
    got, got_s = torch.tensor(want).cuda(), torch.tensor(want_s).cuda()
    blocks.bounds(raw, scales, kind, table, lens, cu, total, size, want, want_s)
    codes, gs = on_gpu(raw, scales, kind)
    q().qcache_bounds(codes, gs, dev(table), dev(lens), got, got_s, cu_q=None if cu is None else dev(cu), total=total)
    assert np.array_equal(got_s.cpu().numpy(), want_s, equal_nan=True)
    assert np.array_equal(got.cpu().numpy(), want)


def test_bounds_clip_what_is_out_of_range():
    rng = np.random.default_rng(3)
    lens = [40, -6, 1 << 30, 96, 10]
    table, pages = tables(rng, [96, 96, 96, 96, 96], 16, width=6)
    raw, scales = cache(rng, "int8", pages, 2, 16, 64)
    codes, gs = on_gpu(raw, scales, "int8")
    for cu in ([0, 9, 3, 12, 30, 20], [-4, 2, 2, 1 << 30, 7, 9], [30, 1, 2, 3, 4, 5], [2, 2, 50, 60, 200, 260]):
        for total in (30, 260):
            want, want_s = np.zeros((pages, 2, 2, 64), np.int8), np.zeros((pages, 2), np.float32)
            got, got_s = q().new_bounds(codes)
            blocks.bounds(raw, scales, "int8", table, lens, cu, total, 16, want, want_s)
            q().qcache_bounds(codes, gs, dev(table), dev(lens), got, got_s, cu_q=dev(cu), total=total)
            assert np.array_equal(got_s.cpu().numpy(), want_s) and np.array_equal(got.cpu().numpy(), want)


# ----------------------------------------------------------------- select ---
SELECT = [  # page size, heads, kv heads, channels, lengths, new tokens, count, first, recent, table width
    (16, 1, 1, 64, [100], None, 3, 1, 1, None), (16, 64, 8, 128, [1000, 17, 5, 400, 800], None, 10, 1, 1, None),
    (64, 5, 5, 128, [3000, 900, 64], None, 7, 2, 3, None), (16, 8, 2, 64, [700, 650], [40, 33], 6, 0, 1, None),
    (32, 34, 2, 128, [2000, 60, 0, 999], [5, 60, 0, 70], 9, 1, 2, None), (16, 14, 2, 64, [6000], [50], 40, 1, 1, None),
    (16, 4, 4, 128, [9000, 300], None, 64, 2, 1, 700), (16, 16, 2, 64, [12000, 70], [20, 3], 33, 1, 4, 800),
    (16, 8, 8, 64, [70000, 3000], None, 100, 1, 1, None), (16, 4, 1, 128, [66000, 40], [35, 40], 17, 1, 1, 4500),
    (16, 8, 2, 64, [30000, 500], [9, 4], 20, 1, 1, 2000), (16, 8, 8, 64, [70000, 3000], None, 100, 1, 1, 8300),
    (16, 8, 1, 64, [500], [480], 2, 1, 1, None), (16, 8, 1, 64, [500], [480], 300, 5, 5, None),
    # one new token each, tables of 257 to 4096 pages and more, more rows than are counted
    (16, 8, 2, 128, [4112, 4097, 4096, 17, 0, 65536], None, 11, 1, 1, 4096), (32, 8, 8, 64, [8256, 130000, 40000], None, 300, 7, 9, 4096),
    (16, 4, 4, 128, [4100] * 30 + [900, 5000], None, 2, 1, 1, 320), (16, 20, 10, 64, [5000, 20, 4200] * 40, None, 5, 0, 1, 330),
    (16, 2, 1, 128, [65600, 300], None, 30, 1, 1, 4110), (64, 8, 1, 64, [262000], None, 4000, 1, 1, 4094)]


@pytest.mark.parametrize("coarse", [False, True])
@pytest.mark.parametrize("case", SELECT, ids=str)
def test_select(coarse, case):
    """coarse: bounds and scales of few values, so that many scores are equal, and pages that are not there."""
    say("select", coarse, case)
    size, hq, heads, dim, lens, new, count, first, recent, width = case
    rng = np.random.default_rng(sum(lens) + count + coarse)
    table, pages = tables(rng, lens, size, width=width, lost=0.05 if coarse else 0.0)
    limits = rng.integers(-1 if coarse else -127, 2 if coarse else 128, (pages, heads, 2, dim)).astype(np.int8)
    steps = rng.uniform(0.01, 0.05, (pages, heads)).astype(np.float32)
    if coarse:
        limits[rng.random(limits.shape[:2]) < 0.5] = 1
        steps[:] = 0.5
        steps[rng.random(steps.shape) < 0.03] = np.nan
        steps[rng.random(steps.shape) < 0.03] = 0.0
    cu = None if new is None else np.r_[0, np.cumsum(new)]
    total = len(lens) if new is None else int(cu[-1])
    x = rows(rng, total, hq, dim)
    if coarse:
        x[0] = 0.0
        x[-1, 0, 3] = float("nan")
        x[total // 2, -1, 1] = float("inf")
    want = blocks.select(f64(x), limits, steps, table, lens, cu, count, size, first, recent)
    got = q().qblock_select(x, torch.tensor(limits).cuda(), torch.tensor(steps).cuda(), dev(table), dev(lens), count, size,
                            cu_q=None if cu is None else dev(cu), first=first, recent=recent)
    assert got.shape == (total, heads, count) and got.dtype is torch.int32
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,width", [(None, 100), (None, 900), (None, 3000), ([20, 3], 100), ([20, 3], 3000)], ids=str)
def test_select_by_queries_whose_sums_pass_float32(dim, new, width):
    """Finite queries rank the pages, however large: 3.3e38 and more together, beside rows of ordinary ones, of
    infinities and of numbers far apart."""
    rng = np.random.default_rng(dim + width)
    size, hq, heads, lens, count = 16, 16, 2, [1590, 1400], 9
    table, pages = tables(rng, lens, size, width=width)
    limits = rng.integers(-127, 128, (pages, heads, 2, dim)).astype(np.int8)
    steps = rng.uniform(0.01, 0.05, (pages, heads)).astype(np.float32)
    cu = None if new is None else np.r_[0, np.cumsum(new)]
    total = 2 if new is None else int(cu[-1])
    x = rows(rng, total, hq, dim)
    x[0] = (x[0] * 1e38).clamp(-3.3e38, 3.3e38)  # some sums pass, of most channels
    x[-1, :, 1] = 3.3e38                         # of one channel; the others count for nothing beside it ...
    x[-1, :, 2:9] = -1e38                        # ... but for these
    assert torch.isfinite(x).all()
    if total > 2:
        x[1] *= 1e38
        x[1, 3, 5] = float("inf")
        x[2] *= torch.tensor(np.exp2(rng.integers(-100, 100, (hq, 1))), device="cuda")
        x[3] *= 1e-38
    want = blocks.select(f64(x), limits, steps, table, lens, cu, count, size, 1, 1)
    assert (want[0, 0, 1:-1] != np.arange(1, count - 1)).any()
    got = q().qblock_select(x, torch.tensor(limits).cuda(), torch.tensor(steps).cuda(), dev(table), dev(lens), count, size,
                            cu_q=None if cu is None else dev(cu))
    assert np.array_equal(got.cpu().numpy(), want)


def test_a_captured_step_over_long_tables():
    """Selection and attention, both split over workgroups and joined by the last, captured, and replayed with other lengths and
    queries, eager calls on the same stream between."""
    rng = np.random.default_rng(21)
    size, hq, heads, dim, batch, width, count = 16, 8, 2, 64, 5, 1200, 24
    pages = batch * width
    table = dev(rng.permutation(pages).reshape(batch, width))
    codes = torch.tensor(rng.integers(0, 256, (pages, 2, heads, size, dim), dtype=np.uint8)).cuda().view(torch.int8)
    scales = torch.tensor(rng.uniform(0.005, 0.02, (pages, 2, heads, size)), dtype=torch.float32).cuda()
    limits, steps = q().new_bounds(codes)
    lens = dev([width * size] * batch)
    cu = np.arange(batch + 1) * width * size
    q().qcache_bounds(codes, scales, table, lens, limits, steps, cu_q=dev(cu), total=int(cu[-1]))
    x = rows(rng, batch, hq, dim)

    def call():
        picks = q().qblock_select(x, limits, steps, table, lens, count, size)
        return picks, q().qattn_blocks(x, codes, scales, table, lens, picks)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        first = call()
        second = call()
    for turn in range(6):
        say("replay", turn)
        have = rng.integers(1, width * size, batch) if turn % 2 else np.array([4096, 4112, 0, 19200, 300])
        lens.copy_(dev(have))
        x.copy_(rows(rng, batch, hq, dim))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
            eager = call()
            graph.replay()
        torch.cuda.synchronize()
        want = blocks.select(f64(x), limits.cpu().numpy(), steps.cpu().numpy(), table.cpu().numpy(), have, None, count, size, 1, 1)
        for picks, out in (first, second, eager):
            assert np.array_equal(picks.cpu().numpy(), want)
            assert torch.equal(out, eager[1])


def test_select_in_several_batches():
    """More scores than the workspace holds at a time."""
    rng = np.random.default_rng(8)
    size, heads, dim, lens, new, count = 16, 16, 64, [80000, 79990], [300, 77], 20
    table, pages = tables(rng, lens, size)
    limits = rng.integers(-127, 128, (pages, heads, 2, dim)).astype(np.int8)
    steps = rng.uniform(0.01, 0.05, (pages, heads)).astype(np.float32)
    cu = np.r_[0, np.cumsum(new)]
    x = rows(rng, int(cu[-1]), heads, dim)
    got = q().qblock_select(x, torch.tensor(limits).cuda(), torch.tensor(steps).cuda(), dev(table), dev(lens), count, size, cu_q=dev(cu)).cpu().numpy()
    # the rows around the batches' ends, and some others; the tile and row kernels' answers for the same rows
    sample = np.unique(np.r_[0, 199:215, 295:305, 376, rng.integers(0, 377, 10)])
    one = [(t, 0 if t < 300 else 1) for t in sample]
    want = blocks.select(f64(x)[sample], limits, steps, table[[b for _, b in one]], [lens[b] - new[b] + 1 + t - cu[b] for t, b in one], None,
                         count, size, 1, 1)
    assert np.array_equal(got[sample], want)


@pytest.mark.parametrize("falls", [False, True])
def test_select_of_many_sequences_in_batches_of_16_rows(falls):
    """Sequences of no row and of up to 40, several to a batch and several batches to one; rows of nobody before, between
    (starts that fall) and behind."""
    rng = np.random.default_rng(31 + falls)
    size, heads, dim, count, width = 16, 32, 64, 4, 66000  # the scores of 16 rows are more than is kept at a time
    new = [0, 3, 1, 16, 17, 0, 0, 5, 40, 2, 1, 1, 31, 0] + [1] * 70 + [0] * 70 + [9]
    lens = [n + int(rng.integers(0, 200)) for n in new]
    cu = 5 + np.r_[0, np.cumsum(new)]
    if falls:
        cu[20], cu[33], cu[90] = 0, cu[40], -7
    total = int(cu.max()) + 6
    table, pages = tables(rng, lens, size, width=width)
    limits = rng.integers(-127, 128, (pages, heads, 2, dim)).astype(np.int8)
    steps = rng.uniform(0.01, 0.05, (pages, heads)).astype(np.float32)
    x = rows(rng, total, heads, dim)
    want = blocks.select(f64(x), limits, steps, table, lens, cu, count, size, 1, 1)
    out = torch.full((total, heads, count), -9, dtype=torch.int32, device="cuda")
    q().qblock_select(x, torch.tensor(limits).cuda(), torch.tensor(steps).cuda(), dev(table), dev(lens), count, size, cu_q=dev(cu), out=out)
    assert np.array_equal(out.cpu().numpy(), want)


def test_select_out_of_range_and_nobodys_rows():
    rng = np.random.default_rng(9)
    lens = [40, -6, 1 << 30, 96, 10]
    table, pages = tables(rng, [96] * 5, 16, width=6)
    limits = rng.integers(-127, 128, (pages, 2, 2, 64)).astype(np.int8)
    steps = rng.uniform(0.01, 0.05, (pages, 2)).astype(np.float32)
    x = rows(rng, 30, 4, 64)
    for cu in ([0, 9, 3, 12, 30, 20], [-4, 2, 2, 1 << 30, 7, 9], [30, 1, 2, 3, 4, 5], [2, 2, 5, 6, 20, 26]):
        for t in (table, np.pad(table, ((0, 0), (0, 800)), constant_values=-1), np.pad(table, ((0, 0), (0, 5000)), constant_values=-1)):
            if t is not table:
                lens[2] = 96
            want = blocks.select(f64(x), limits, steps, t, lens, cu, 3, 16, 1, 1)
            out = torch.full((32, 2, 3), -9, dtype=torch.int32, device="cuda")
            q().qblock_select(x, torch.tensor(limits).cuda(), torch.tensor(steps).cuda(), dev(t), dev(lens), 3, 16, cu_q=dev(cu), out=out[:30])
            assert np.array_equal(out[:30].cpu().numpy(), want) and (out[30:] == -9).all()
            lens[2] = 1 << 30


# -------------------------------------------------------------- attention ---
def check_attention(rng, got, x, raw, scales, kind, table, lens, cu, picks, size, hq, heads, sample=None):
    total, _, dim = x.shape
    pages = raw.shape[0]
    xf, scale = f64(x), 1 / math.sqrt(dim)
    have = f64(got)
    for t, b, pos in blocks.rows_of(lens, cu, total, table.shape[1] * size):
        if sample is not None and t not in sample:
            continue
        for h in range(heads):
            at = blocks.tokens_of(picks[t, h], size, pos, table[b], pages)
            page, place = (table[b][at // size], at % size) if len(at) else (np.zeros(0, int), np.zeros(0, int))
            k, v = (ref.code_values(raw[page, w, h, place], kind) * scales[page, w, h, place].astype(np.float64)[:, None] for w in (0, 1))
            for g in range(h * (hq // heads), (h + 1) * (hq // heads)):
                want, bound = ref.attend(xf[t, g], k, v, np.arange(len(at)), scale, weight_error=2.0 ** -16)
                if np.isnan(want).any():
                    assert not np.isfinite(have[t, g][np.isnan(want)]).any()
                    continue
                off = np.abs(have[t, g] - want) - bound
                assert np.all(off <= 0), (t, g, off.max())


ATTEND = [  # page size, heads, kv heads, channels, lengths, new tokens, count
    (16, 1, 1, 64, [1], None, 1), (16, 64, 8, 128, [1000], None, 12), (64, 8, 1, 64, [4000, 100, 64, 65], None, 9),
    (16, 34, 2, 128, [300, 90], None, 5), (32, 5, 5, 128, [500, 40], [9, 40], 4), (256, 6, 2, 64, [900, 255], [7, 200], 2),
    (16, 8, 2, 128, [400], [390], 6), (128, 4, 4, 64, [700, 300, 0], [300, 290, 0], 3), (16, 128, 2, 64, [90, 33], [20, 17], 4),
    (16, 32, 32, 128, [60, 80, 7], [60, 11, 7], 3), (64, 16, 2, 128, [30000], None, 200),
    # more than 512 items of up to 4, 8 and 16 queries, and more than 2048
    (16, 8, 4, 128, [300, 77], [140, 60], 7), (16, 28, 4, 64, [260, 70], [150, 70], 5), (32, 18, 2, 64, [333], [320], 3),
    (16, 4, 4, 128, [500], [200], 9), (16, 16, 4, 64, [700, 20], [510, 20], 4), (32, 12, 4, 128, [40, 620], [40, 490], 5),
    (16, 24, 4, 64, [800], [600], 6), (16, 32, 4, 128, [650, 9], [560, 9], 5), (16, 64, 4, 64, [560, 1], [530, 1], 5),
    (32, 72, 4, 128, [310, 45], [260, 40], 4), (64, 6, 6, 64, [1000], [400], 6)]


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("case", ATTEND, ids=str)
def test_attention(kind, case):
    say("attend", kind, case)
    size, hq, heads, dim, lens, new, count = case
    rng = np.random.default_rng(sum(lens) + count)
    table, pages = tables(rng, lens, size, lost=0.04 if len(lens) > 1 else 0.0)
    raw, scales = cache(rng, kind, pages, heads, size, dim)
    cu = None if new is None else np.r_[0, np.cumsum(new)]
    total = len(lens) if new is None else int(cu[-1])
    x = rows(rng, total, hq, dim)
    # any order, some twice, some of no page, some behind the row
    picks = rng.integers(-1, table.shape[1] + 1, (total, heads, count)).astype(np.int32)
    if len(lens) == 1:  # as a selection gives them
        for t, b, pos in blocks.rows_of(lens, cu, total, table.shape[1] * size):
            seen = pos // size + 1
            for h in range(heads):
                mine = np.sort(rng.permutation(seen)[:count])
                picks[t, h] = np.r_[mine, [-1] * (count - len(mine))]
    # what a row does not see has no influence, whatever it is
    for b, n in enumerate(lens):
        p = table[b, n // size] if n % size else -1
        if 0 <= p < pages:
            scales[p, :, :, n % size:] = np.nan
            raw[p, :, :, n % size:] = 0x7F
    codes, gs = on_gpu(raw, scales, kind)
    got = q().qattn_blocks(x, codes, gs, dev(table), dev(lens), dev(picks), cu_q=None if cu is None else dev(cu))
    sample = None if total <= 70 else set(np.r_[0, total - 1, rng.integers(0, total, 40)].tolist())
    check_attention(rng, got, x, raw, scales, kind, table, lens, cu, picks, size, hq, heads, sample)
    again = q().qattn_blocks(x, codes, gs, dev(table), dev(lens), dev(picks), cu_q=None if cu is None else dev(cu))
    assert torch.equal(got, again)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("n,new", [(900, 1), (900, 40), (5000, 1)])
def test_every_page_is_all_of_the_cache(kind, n, new):
    """With every page picked the outputs are qattn_cache's, up to the order of the sums: both inside the same bound."""
    rng = np.random.default_rng(n + new)
    size, hq, heads, dim, lens = 16, 16, 2, 128, [n, n // 2]
    table, pages = tables(rng, lens, size)
    raw, scales = cache(rng, kind, pages, heads, size, dim)
    codes, gs = on_gpu(raw, scales, kind)
    cu = np.array([0, new, 2 * new])
    x = rows(rng, 2 * new, hq, dim)
    limits, steps = q().new_bounds(codes)
    q().qcache_bounds(codes, gs, dev(table), dev(lens), limits, steps, cu_q=dev([0] + np.cumsum(lens).tolist()), total=sum(lens))
    count = table.shape[1]
    picks = q().qblock_select(x, limits, steps, dev(table), dev(lens), count, size, cu_q=dev(cu))
    sparse = q().qattn_blocks(x, codes, gs, dev(table), dev(lens), picks, cu_q=dev(cu))
    full = q().qattn_cache(x, codes, gs, dev(table), dev(lens), cu_q=dev(cu))
    # 2^-8 of the output each, weights of 2^-16 of the values' size, scores and sums in fp32 over n keys
    size_of = float(torch.tensor(scales).max()) * (128 if kind == "int8" else 448)
    off = (sparse.float() - full.float()).abs()
    assert (off <= 2 * 2.0 ** -8 * full.float().abs() + 2 * size_of * (2.0 ** -16 + (n + 64) * 2.0 ** -23 + 4 * dim * 2.0 ** -24 * 40) + 1e-37).all()


def test_counts_every_key_once():
    """With q = 0 every weight is one; values of one in one channel: an output is the share of the row's keys that have theirs there."""
    rng = np.random.default_rng(14)
    size, heads, dim = 16, 2, 64
    for lens, new, count in (([3000], [1], 100), ([700, 333], [5, 9], 30), ([900], [600], 11), ([2000, 2000], [1, 1], 125)):
        table, pages = tables(rng, lens, size)
        cu = np.r_[0, np.cumsum(new)]
        total = int(cu[-1])
        picks = np.full((total, heads, count), -1, np.int32)
        for t, b, pos in blocks.rows_of(lens, cu, total, table.shape[1] * size):
            for h in range(heads):
                mine = np.sort(rng.permutation(pos // size + 1)[:count])
                picks[t, h, :len(mine)] = mine
        x = torch.zeros(total, 2 * heads, dim, dtype=torch.bfloat16, device="cuda")
        most = max(lens)
        parts = ref.counting_parts(most, dim)
        for part in range(parts):
            values = ref.counting_values(most, dim, part, parts)
            raw = np.ones((pages, 2, heads, size, dim), np.uint8)
            for b, n in enumerate(lens):
                at = np.arange(n)
                raw[table[b][at // size], 1, :, at % size] = values[at][:, None]
            codes, gs = on_gpu(raw, np.ones((pages, 2, heads, size), np.float32), "int8")
            got = f64(q().qattn_blocks(x, codes, gs, dev(table), dev(lens), dev(picks), cu_q=dev(cu)))
            for t, b, pos in blocks.rows_of(lens, cu, total, table.shape[1] * size):
                for h in range(heads):
                    seen = np.zeros((1, most))
                    seen[0, blocks.tokens_of(picks[t, h], size, pos, table[b], pages)] = 1
                    assert not ref.miscounted(got[t, 2 * h:2 * h + 2], np.repeat(seen, 2, 0), values).any(), (t, h)


def test_nan_in_what_a_row_sees():
    """A NaN code or scale among the picked pages' seen tokens shows; in other pages or behind the row it does not."""
    rng = np.random.default_rng(15)
    size, heads, dim, lens = 16, 2, 128, [100]
    table, pages = tables(rng, lens, size)
    raw, scales = cache(rng, "e4m3", pages, heads, size, dim)
    x = rows(rng, 1, 4, dim)
    picks = np.array([[[0, 2, 6], [1, 2, 6]]], np.int32)
    raw[table[0, 1], 1, 0, 5, 7] = 0xFF     # page 1, head 0: not picked by head 0
    raw[table[0, 6], 1, 0, 3, 9] = 0x7F     # token 99: seen by head 0 in channel 9
    raw[table[0, 6], 0, 1, 4] = 0x7F        # token 100: behind the row
    scales[table[0, 6], 1, 1, 5] = np.nan
    codes, gs = on_gpu(raw, scales, "e4m3")
    got = q().qattn_blocks(x, codes, gs, dev(table), dev(lens), dev(picks)).float()
    bad = torch.zeros(1, 4, dim, dtype=torch.bool, device="cuda")
    bad[0, :2, 9] = True
    assert torch.equal(~torch.isfinite(got), bad)


def test_rows_behind_and_rows_that_see_nothing():
    rng = np.random.default_rng(16)
    size, heads, dim = 16, 2, 64
    lens = [40, -6, 1 << 30, 96, 2]
    table, pages = tables(rng, [96] * 5, size, width=6)
    raw, scales = cache(rng, "int8", pages, heads, size, dim)
    codes, gs = on_gpu(raw, scales, "int8")
    x = rows(rng, 30, 4, dim)
    picks = rng.integers(-3, 9, (30, heads, 4)).astype(np.int32)
    picks[3] = -1
    for cu in ([0, 9, 3, 12, 30, 20], [-4, 2, 2, 1 << 30, 7, 9], [30, 1, 2, 3, 4, 5], [2, 2, 5, 6, 20, 26]):
        out = torch.full((33, 4, dim), 5.0, dtype=torch.bfloat16, device="cuda")
        q().qattn_blocks(x, codes, gs, dev(table), dev(lens), dev(picks), cu_q=dev(cu), out=out[:30])
        check_attention(rng, out[:30], x, raw, scales, "int8", table, lens, cu, picks, size, 4, heads)
        mine = {t for t, _, _ in blocks.rows_of(lens, cu, 30, 96)}
        others = [t for t in range(33) if t not in mine]
        assert (out[others] == 5).all()
    none = q().qattn_blocks(x[:5], codes, gs, dev(table), dev([0] * 5), dev(picks[:5]))
    assert (none == 0).all()
    empty = q().new_cache(0, size, heads, dim)
    assert (q().qattn_blocks(x[:5], *empty, dev(table), dev(lens), dev(picks[:5])) == 0).all()


def test_strided_queries():
    rng = np.random.default_rng(17)
    size, heads, dim, lens = 16, 2, 64, [200, 150]
    table, pages = tables(rng, lens, size)
    raw, scales = cache(rng, "int8", pages, heads, size, dim)
    codes, gs = on_gpu(raw, scales, "int8")
    limits, steps = q().new_bounds(codes)
    q().qcache_bounds(codes, gs, dev(table), dev(lens), limits, steps, cu_q=dev([0, 200, 350]), total=350)
    fused = rows(rng, 2, 12, dim)
    x = fused[:, 2:6]
    for view in (x, x.transpose(0, 1).contiguous().transpose(0, 1)):
        a = q().qblock_select(view, limits, steps, dev(table), dev(lens), 5, size)
        b = q().qblock_select(x.contiguous(), limits, steps, dev(table), dev(lens), 5, size)
        assert torch.equal(a, b)
        assert torch.equal(q().qattn_blocks(view, codes, gs, dev(table), dev(lens), a),
                           q().qattn_blocks(x.contiguous(), codes, gs, dev(table), dev(lens), a))


def test_a_long_cache_past_32_bits():
    """Codes of more than 2^32 bytes: pages at the far end are read from where they are."""
    size, heads, dim = 64, 8, 128
    pages = (1 << 32) // (2 * heads * size * dim) + 40
    codes = torch.zeros(pages, 2, heads, size, dim, dtype=torch.int8, device="cuda")
    scales = torch.ones(pages, 2, heads, size, device="cuda")
    far = pages - 20
    codes[far, 1] = 3
    codes[far, 0] = 1
    codes[far + 1, 1] = 5
    table = torch.full((1, 30), far + 1, dtype=torch.int32, device="cuda")
    table[0, 3] = far
    table[0, 7] = 11
    lens = dev([30 * size])
    x = torch.ones(1, 16, dim, dtype=torch.bfloat16, device="cuda")
    limits, steps = q().new_bounds(codes)
    q().qcache_bounds(codes, scales, table, lens, limits, steps, cu_q=dev([0, 30 * size]), total=30 * size)
    assert (limits[far] == 127).all() and (steps[far + 1] == 0).all()
    picks = q().qblock_select(x, limits, steps, table, lens, 3, size)
    assert (picks == torch.tensor([0, 3, 29], device="cuda")).all()
    got = q().qattn_blocks(x, codes, scales, table, lens, picks)
    # page 3's scores are 128 / sqrt(128) above the others': their weight is exp(-11.3)
    w = math.exp(-math.sqrt(128))
    want = (3 + 2 * 5 * w) / (1 + 2 * w)
    assert (got.float() - want).abs().max() <= want * (2.0 ** -8 + 2.0 ** -14)


def test_replay_and_other_streams():
    """Bounds, selection and attention captured and replayed with other contents, eager work between, and on a stream of their own."""
    rng = np.random.default_rng(18)
    size, heads, hq, dim, width = 16, 2, 16, 64, 60
    pages = 3 * width
    codes = torch.zeros(pages, 2, heads, size, dim, dtype=torch.int8, device="cuda")
    scales = torch.zeros(pages, 2, heads, size, device="cuda")
    limits, steps = q().new_bounds(codes)
    table, lens, cu = torch.zeros(3, width, dtype=torch.int32, device="cuda"), dev([0] * 3), dev([0] * 4)
    x = torch.zeros(12, hq, dim, dtype=torch.bfloat16, device="cuda")

    def call():
        q().qcache_bounds(codes, scales, table, lens, limits, steps, cu_q=cu, total=12)
        picks = q().qblock_select(x, limits, steps, table, lens, 8, size, cu_q=cu)
        return picks, q().qattn_blocks(x, codes, scales, table, lens, picks, cu_q=cu)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = call()
    for _ in range(4):
        codes.random_(-127, 128)
        scales.uniform_(0.005, 0.02)
        limits.random_(-127, 128)
        steps.uniform_(0.1, 0.2)
        table.copy_(dev(rng.permutation(pages).reshape(3, width)))
        lens.copy_(dev(rng.integers(12, width * size, 3)))
        cu.copy_(dev(np.r_[0, np.sort(rng.integers(0, 13, 2)), 12]))
        x.normal_()
        start = limits.clone(), steps.clone()
        results = []
        for run in ("replay", "eager", "side"):
            limits.copy_(start[0]), steps.copy_(start[1])
            torch.cuda.synchronize()
            if run == "replay":
                graph.replay()
                got = out
            elif run == "eager":
                got = call()
            else:
                with torch.cuda.stream(side):
                    got = call()
            torch.cuda.synchronize()
            results.append([t.clone() for t in got] + [limits.clone(), steps.clone()])
        for other in results[1:]:
            assert all(torch.equal(a, b) for a, b in zip(results[0], other))


def test_refusals():
    codes, scales = q().new_cache(8, 16, 2, 64)
    limits, steps = q().new_bounds(codes)
    table, lens = dev([[0, 1, 2]] * 2), dev([5, 6])
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    picks = torch.zeros(2, 2, 3, dtype=torch.int32, device="cuda")
    for bad in (lambda: q().qcache_bounds(codes, scales, table, lens, limits[:4], steps[:4]), lambda: q().qcache_bounds(codes, scales, table, lens, limits, steps[:4]),
                lambda: q().qcache_bounds(codes, scales, table, lens, limits, steps, cu_q=dev([0, 1, 2])),
                lambda: q().qcache_bounds(codes, scales, table, lens, limits, steps, total=5),
                lambda: q().qblock_select(x[:1], limits, steps, table, lens, 3, 16), lambda: q().qblock_select(x[:, :3], limits, steps, table, lens, 3, 16),
                lambda: q().qblock_select(x, limits, steps, table, lens, 1, 16), lambda: q().qblock_select(x, limits, steps, table, lens, 3, 16, recent=0),
                lambda: q().qblock_select(x, limits, steps, table, lens, 3, 16, out=picks[:1]),
                lambda: q().qblock_select(x, limits.transpose(2, 3), steps, table, lens, 3, 16),
                lambda: q().qattn_blocks(x, codes, scales, table, lens, picks[:, :1]), lambda: q().qattn_blocks(x, codes, scales, table, lens, picks[0]),
                lambda: q().qattn_blocks(x, codes, scales, table, lens, picks, out=x.float())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q().qcache_bounds(codes, scales, table, lens, limits.view(torch.uint8), steps), lambda: q().qblock_select(x.float(), limits, steps, table, lens, 3, 16),
                lambda: q().qattn_blocks(x, codes, scales, table, lens, picks.long()), lambda: q().qblock_select(x, limits, steps, table.long(), lens, 3, 16)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: q().qblock_select(x, limits, steps, table, lens, 3, 24), lambda: q().qattn_blocks(x, codes, scales, table, lens, picks, sm_scale=-1.0),
                lambda: q().qattn_blocks(x, codes, scales, table, lens, picks[:, :, :0])):
        with pytest.raises(q().Qw3Error) as e:
            bad()
        assert e.value.status == q().QW3_ERR_SHAPE
