"""The calls on the cache's pages on the GPU against oracle/pages.py: every
number and every byte equal."""
import sys

import numpy as np
import pytest
import torch

from oracle import pages as ref

pytestmark = pytest.mark.gpu

TORCH = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def q():
    import dequant_gemv_qgemv_amd as mod
    return mod


def say(*args):
    print("[gpu-case]", *args, file=sys.stderr, flush=True)


def dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def same(got, want):
    assert np.array_equal(got.cpu().numpy(), want)


def random_tables(rng, batch, width, size, spare, shared=0.3, bad=0.05):
    """(refs, table, lens): sequences of any length, some entries shared with others, some that name no page."""
    lens = rng.integers(0, width * size + 1, batch)
    lens[rng.random(batch) < 0.1] = 0
    table = np.full((batch, width), -1, np.int64)
    at = 0
    for b in range(batch):
        held = min(width, -(-int(lens[b]) // size) + int(rng.integers(0, 2)))
        table[b, :held] = np.arange(at, at + held)
        at += held
        if b and rng.random() < shared:  # follows another as far as both reach
            other = int(rng.integers(0, b))
            n = min(held, int((table[other] >= 0).sum()))
            table[b, :n] = table[other, :n]
    used = np.unique(table[table >= 0])
    pages = len(used) + spare
    names = rng.permutation(pages)
    table = np.where(table >= 0, names[np.searchsorted(used, np.maximum(table, 0)).clip(max=max(pages - 1, 0))] if pages else -1, -1)
    refs = np.bincount(table[table >= 0], minlength=pages)
    lost = rng.random(table.shape) < bad
    table[lost] = rng.choice([-1, -7, pages, 2 ** 31 - 1], lost.sum())
    return refs.astype(np.int32), table.astype(np.int32), lens.astype(np.int32)


def check_reserve(refs, table, lens, cu, total, size):
    """One call against the oracle; the tensors as they are after it."""
    r, t = dev(refs), dev(table)
    got = q().qcache_reserve(r, t, dev(lens), size, cu=None if cu is None else dev(cu), total=None if cu is None else total)
    r1, t1 = refs.copy(), table.copy()
    want = ref.reserve(r1, t1, lens, cu, total, size)
    for g, w in zip(got + (r, t), want + (r1, t1)):
        same(g, w)
    return got


@pytest.mark.parametrize("size", [16, 64])
@pytest.mark.parametrize("batch,width,spare", [(1, 1, 0), (1, 3, 2), (4, 5, 3), (33, 9, 200), (33, 9, 11), (257, 4, 300), (1030, 3, 900),
                                               (2500, 2, 5000), (2, 600, 700)])
def test_reserve(size, batch, width, spare):
    say("reserve", size, batch, width, spare)
    rng = np.random.default_rng(batch + width + spare + size)
    for k in range(4):
        refs, table, lens = random_tables(rng, batch, width, size, spare)
        check_reserve(refs, table, lens, None, batch, size)
        new = rng.integers(0, 1 + [1, 3, 3 * size, width * size][k], batch)
        cu = np.r_[0, np.cumsum(new)]
        total = int(cu[-1])
        check_reserve(refs, table, lens, cu, total, size)
        check_reserve(refs, table, lens, cu + 2, total + 5, size)  # rows before the first and behind the last are nobody's


def test_reserve_clips_what_is_out_of_range():
    rng = np.random.default_rng(5)
    refs, table, lens = random_tables(rng, 6, 4, 16, 20)
    lens[1], lens[3] = -5, 1 << 30
    for cu in ([0, 9, 3, 12, 12, 40, 20], [-4, 2, 2, 1 << 30, 7, 9, 30], [30, 1, 2, 3, 4, 5, 6], [0] * 7):
        check_reserve(refs, table, lens, np.array(cu), 30, 16)
    check_reserve(refs[:0], table, lens, None, 6, 16)       # no pages at all
    check_reserve(refs, table[:, :0], lens, None, 6, 16)    # no entries
    slots, lens_out, copies = q().qcache_reserve(dev(refs), dev(table[:0]), dev(lens[:0]), 16, cu=dev([0]), total=3)
    assert (slots == -1).all() and slots.shape == (3,) and lens_out.shape == (0,) and copies.shape == (0, 2)


def test_reserve_many_sequences_with_starts_that_fall():
    rng = np.random.default_rng(6)
    refs, table, lens = random_tables(rng, 2300, 3, 16, 1500)
    cu = np.cumsum(rng.integers(-3, 6, 2301))
    check_reserve(refs, table, lens, cu, int(cu.max()) + 4, 16)


@pytest.mark.parametrize("batch,out,width,size", [(1, 1, 1, 16), (4, 4, 5, 16), (7, 30, 9, 64), (96, 96, 300, 16), (3, 2, 9001, 16), (50, 0, 4, 16),
                                                  (0, 3, 4, 32)])
def test_fork(batch, out, width, size):
    say("fork", batch, out, width, size)
    rng = np.random.default_rng(batch + out + width)
    refs, table, lens = random_tables(rng, batch, width, size, 7) if batch else (np.zeros(9, np.int32), np.zeros((0, width), np.int32), np.zeros(0, np.int32))
    if batch > 3:
        lens[1], lens[2] = -3, 1 << 30
    parents = rng.integers(-1, batch + 1, out).astype(np.int32)
    r = dev(refs)
    got = q().qcache_fork(r, dev(table).view(batch, width), dev(lens), dev(parents), size)
    want = ref.fork(refs, table, lens, parents, size)
    for g, w in zip(got + (r,), want + (refs,)):
        same(g, w)


def random_layers(rng, kind, layers, pages, heads, page, dim):
    raw = torch.tensor(rng.integers(0, 256, (layers, pages, 2, heads, page, dim)), dtype=torch.uint8)
    scales = torch.tensor(rng.standard_normal((layers, pages, 2, heads, page)), dtype=torch.float32)
    return raw.cuda().view(TORCH[kind]), scales.cuda()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("layers,pages,heads,page,dim", [(1, 5, 1, 16, 64), (3, 40, 3, 16, 128), (2, 9, 8, 64, 128), (1, 4, 5, 256, 64)])
def test_copy(kind, layers, pages, heads, page, dim):
    say("copy", kind, layers, pages, heads, page, dim)
    rng = np.random.default_rng(pages + dim)
    codes, scales = random_layers(rng, kind, layers, pages, heads, page, dim)
    ids = rng.permutation(pages)
    copies = [(ids[0], ids[1]), (-1, -1), (ids[0], ids[2]), (ids[3], ids[3]), (ids[3], pages), (-1, ids[3]), (1 << 30, ids[3])]
    want_c, want_s = codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy()
    ref.copy(want_c, want_s, copies)
    q().qcache_copy(codes, scales, dev(copies))
    same(codes.view(torch.uint8), want_c)
    same(scales, want_s)
    # one layer of them, as a cache of its own
    copies = [(ids[1], ids[0])]
    ref.copy(want_c[-1:], want_s[-1:], copies)
    q().qcache_copy(codes[-1], scales[-1], dev(copies))
    same(codes.view(torch.uint8), want_c)
    same(scales, want_s)


# layers, heads, page, dim, lengths, new tokens: up to 512 for each sequence on average in one workgroup for each head, more by all of the card
COMPACT = [(1, 1, 16, 64, [1], [1]), (2, 3, 16, 128, [40, 16, 0, 7], [13, 16, 0, 7]), (1, 2, 64, 128, [700, 300, 90], [600, 256, 64]),
           (1, 8, 16, 64, [300, 20, 900, 33], [257, 5, 700, 33]), (2, 2, 32, 128, [1500], [1500]), (1, 3, 16, 64, [2000, 5, 0, 700], [1999, 5, 0, 700]),
           (3, 1, 16, 128, [17000, 300], [16999, 120]), (2, 5, 64, 128, [9000, 40, 5000], [8000, 40, 4999]), (1, 11, 16, 64, [4000], [3990])]


@pytest.mark.parametrize("share", [0.0, 0.04, 0.5, 0.97, 1.0])
@pytest.mark.parametrize("case", COMPACT, ids=str)
def test_compact(case, share):
    say("compact", case, share)
    layers, heads, page, dim, lens, new = case
    rng = np.random.default_rng(sum(lens))
    width = max(-(-n // page) for n in lens) + 1
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    ids = rng.permutation(pages)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    codes, scales = random_layers(rng, "int8", layers, pages, heads, page, dim)
    keep = rng.random(sum(new) + 3) < share
    cu = np.r_[0, np.cumsum(new)]
    if len(lens) > 2:
        table[0, width // 3] = -1  # tokens without a page come out as zeros
        table[-1, 0] = pages
    for layer in (None, layers - 1):
        c, s = (codes, scales) if layer is None else (codes[layer], scales[layer])
        want_c, want_s = codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy()
        part = slice(None) if layer is None else slice(layer, layer + 1)
        want = ref.compact(want_c[part], want_s[part], table, lens, keep, cu, page)
        got = q().qcache_compact(c, s, dev(table), dev(lens), dev(keep, torch.bool if layer is None else torch.uint8), cu_q=dev(cu))
        same(got, want)
        same(codes.view(torch.uint8), want_c)
        same(scales, want_s)


def test_compact_out_of_range():
    """Starts that fall, lengths below the new tokens and above the table, one token each without starts."""
    rng = np.random.default_rng(9)
    page, pages, width = 16, 40, 6
    lens = np.array([50, 3, 96, -4, 1 << 30, 20], np.int32)
    table = rng.permutation(pages)[:36].reshape(6, width).astype(np.int32)
    for cu in (np.array([0, 9, 30, 12, 60, 61, 70]), np.array([-5, 20, 20, 90, 7, 1 << 30, 3]), None):
        for extra in (0, 4000):  # the second by all of the card: room for rows that nobody has
            if cu is None and extra:
                continue
            keep = rng.random(75 + extra if cu is not None else 6) < 0.6
            codes, scales = random_layers(rng, "e4m3", 1, pages, 2, page, 64)
            want_c, want_s = codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy()
            want = ref.compact(want_c, want_s, table, lens, keep, cu, page)
            got = q().qcache_compact(codes, scales, dev(table), dev(lens), dev(keep, torch.bool), cu_q=None if cu is None else dev(cu))
            same(got, want)
            same(codes.view(torch.uint8), want_c)
            same(scales, want_s)


def test_compact_any_bytes_captured_and_replayed():
    """By all of the card: keep of any values at any address, more tokens than there are; a graph with other contents."""
    rng = np.random.default_rng(20)
    page, width, heads, dim, rows = 64, 160, 2, 64, 11001
    pages = 2 * width
    table = rng.permutation(pages).reshape(2, width).astype(np.int32)
    codes, scales = random_layers(rng, "int8", 1, pages, heads, page, dim)
    pool = torch.zeros(rows + 40, dtype=torch.uint8, device="cuda")
    lens, cu, t = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"), dev(table)
    for skew in (0, 1, 7, 15, 16, 23):
        keep = pool[skew:skew + rows]

        def call():
            return q().qcache_compact(codes, scales, t, lens, keep, cu_q=cu)

        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = call()
        for have, starts in (([10240, 4000], [0, 8000, 11001]), ([2047, 900], [3, 6001, 10990]), ([9000, 3000], [0, 8193, 11001])):
            say("compact", skew, have, starts)
            bytes_ = np.where(rng.random(rows) < 0.5, 0, rng.choice([1, 2, 127, 128, 255], rows)).astype(np.uint8)
            keep.copy_(torch.tensor(bytes_))
            lens.copy_(dev(have))
            cu.copy_(dev(starts))
            want_c, want_s = codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy()
            want = ref.compact(want_c, want_s, table, have, bytes_, np.array(starts), page)
            graph.replay()
            same(out, want)
            same(codes.view(torch.uint8), want_c)
            same(scales, want_s)


@pytest.mark.parametrize("share", [0.02, 0.6, 0.999])
def test_compact_many_heads(share):
    """Units of several groups of heads, by far more of them than run at a time."""
    rng = np.random.default_rng(10)
    layers, heads, page, dim, n = 3, 40, 64, 128, 8000
    pages = n // page
    codes = torch.randint(0, 256, (layers, pages, 2, heads, page, dim), dtype=torch.uint8, device="cuda")
    scales = torch.randn(layers, pages, 2, heads, page, device="cuda")
    table = rng.permutation(pages)[None].astype(np.int32)
    keep = rng.random(n) < share
    order = torch.tensor(np.flatnonzero(keep), device="cuda")
    rows = dev(table[0]).long()
    want_c, want_s = codes.clone(), scales.clone()
    to = torch.arange(len(order), device="cuda")
    want_c[:, rows[to // page], :, :, to % page] = codes[:, rows[order // page], :, :, order % page]
    want_s[:, rows[to // page], :, :, to % page] = scales[:, rows[order // page], :, :, order % page]
    got = q().qcache_compact(codes.view(torch.int8), scales, dev(table), dev([n]), dev(keep, torch.bool), cu_q=dev([0, n]))
    assert got.tolist() == [len(order)]
    assert torch.equal(codes, want_c) and torch.equal(scales, want_s)


def test_compact_in_several_launches():
    """More units than a launch has: a cache of 1024 layers, and rows of no sequence behind the two that there are."""
    rng = np.random.default_rng(19)
    layers, heads, page, dim, lens, new, rows = 1024, 1, 16, 64, [420, 300], [410, 300], (1 << 20) + 600
    pages = 50
    table = rng.permutation(pages)[:48].reshape(2, 24).astype(np.int32)
    table = np.pad(table, ((0, 0), (0, 4)), constant_values=-1)
    raw = rng.integers(0, 256, (1, pages, 2, heads, page, dim), dtype=np.uint8)
    floats = rng.standard_normal((1, pages, 2, heads, page)).astype(np.float32)
    codes = torch.tensor(raw).cuda().repeat(layers, 1, 1, 1, 1, 1) ^ (torch.arange(layers, device="cuda") % 256).to(torch.uint8).view(-1, 1, 1, 1, 1, 1)
    scales = torch.tensor(floats).cuda() + torch.arange(layers, device="cuda").view(-1, 1, 1, 1, 1)
    keep = rng.random(rows) < 0.5
    cu = np.r_[0, np.cumsum(new)]
    want_c, want_s = codes.cpu().numpy(), scales.cpu().numpy()
    want = ref.compact(want_c, want_s, table, lens, keep, cu, page)
    got = q().qcache_compact(codes.view(torch.int8), scales, dev(table), dev(lens), dev(keep, torch.bool), cu_q=dev(cu))
    same(got, want)
    same(codes, want_c)
    same(scales, want_s)


def test_life_of_sequences():
    """Reserve, write, fork, reserve with copies, drop drafts, end: every sequence reads back the tokens it was given, and at
    the end all pages are free."""
    rng = np.random.default_rng(11)
    page, heads, dim, pages = 16, 2, 64, 120
    codes, scales = q().new_cache(pages, page, heads, dim)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    table = torch.full((3, 12), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    held = [[], [], []]  # the tokens of each sequence, by number

    def rows(tokens):
        """Keys of a token: its number in the largest channel and in the sign pattern, so that it is read back exactly."""
        x = torch.zeros(len(tokens), heads, dim, device="cuda")
        t = torch.tensor(tokens, device="cuda")
        x[:, :, 0] = 127.0
        x[:, :, 1] = (t % 100).float()[:, None]
        x[:, :, 2] = (t // 100).float()[:, None]
        return x

    def extend(new):
        nonlocal lens, number
        cu = np.r_[0, np.cumsum(new)]
        slots, lens, copies = q().qcache_reserve(refs, table, lens, page, cu=dev(cu), total=int(cu[-1]))
        q().qcache_copy(codes, scales, copies)
        tokens = list(range(number, number + int(cu[-1])))
        number += len(tokens)
        assert (slots >= 0).all() and len(set(slots.tolist())) == len(tokens)
        x = rows(tokens)
        q().qcache_write(x, -x, slots, codes, scales)
        for b, n in enumerate(new):
            held[b] += tokens[cu[b]:cu[b + 1]]

    def check():
        cu = np.r_[0, np.cumsum([len(h) for h in held])]
        assert lens.tolist() == [len(h) for h in held]
        k, v = q().qcache_read(codes, scales, table, dev(cu), int(cu[-1]))
        want = rows(sum(held, [])).to(torch.bfloat16)
        assert torch.equal(k, want) and torch.equal(v, -want)
        names = table[table >= 0].cpu().numpy()
        assert np.array_equal(refs.cpu().numpy(), np.bincount(names, minlength=pages))

    number = 1
    extend([40, 5, 64])
    check()
    for step in range(12):
        parents = rng.integers(0, len(held), int(rng.integers(2, 8)))
        table, lens = q().qcache_fork(refs, table, lens, dev(parents), page)
        held = [list(held[p]) for p in parents]
        check()
        new = rng.integers(0, 7, len(held)).tolist()
        extend(new)
        check()
        keep = rng.random(sum(new)) < 0.5  # of the drafts just written
        cu = np.r_[0, np.cumsum(new)]
        lens = q().qcache_compact(codes, scales, table, lens, dev(keep, torch.bool), cu_q=dev(cu))
        held = [h[:len(h) - n] + [t for t, k in zip(h[len(h) - n:], keep[cu[b]:cu[b + 1]]) if k] for b, (h, n) in enumerate(zip(held, new))]
        check()
    table, lens = q().qcache_fork(refs, table, lens, dev([-1]), page)
    assert (refs == 0).all() and (table == -1).all() and lens.tolist() == [0]


def test_replay():
    """Reserve, fork and compact captured and replayed with other contents, eager work between."""
    rng = np.random.default_rng(12)
    page, width = 16, 6
    codes, scales = random_layers(rng, "int8", 2, 200, 2, page, 64)
    keep = torch.zeros(40, dtype=torch.bool, device="cuda")
    parents = torch.zeros(8, dtype=torch.int32, device="cuda")
    cu = torch.zeros(9, dtype=torch.int32, device="cuda")
    refs = torch.zeros(200, dtype=torch.int32, device="cuda")
    table = torch.full((8, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(8, dtype=torch.int32, device="cuda")

    def call():
        t, n = q().qcache_fork(refs, table, lens, parents, page)
        slots, n, copies = q().qcache_reserve(refs, t, n, page, cu=cu, total=40)
        q().qcache_copy(codes, scales, copies)
        return t, slots, copies, q().qcache_compact(codes, scales, t, n, keep, cu_q=cu)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for _ in range(4):
        r, t, n = random_tables(rng, 8, width, page, 60, bad=0.0)
        n = np.minimum(n, width * page - 6)
        new = rng.integers(0, 6, 8)
        inputs = (np.pad(r, (0, 200 - len(r))), t, n, rng.integers(-1, 8, 8), np.r_[0, np.cumsum(new)], rng.random(40) < 0.5)
        start = codes.clone(), scales.clone()
        results = []
        for run in (graph.replay, call):
            codes.copy_(start[0]), scales.copy_(start[1])
            for to, x in zip((refs, table, lens, parents, cu, keep), inputs):
                to.copy_(torch.tensor(np.asarray(x)).to(to.dtype))
            got = run()
            torch.cuda.synchronize()
            results.append([x.clone() for x in (got or out)] + [refs.clone(), codes.clone(), scales.clone()])
        assert all(torch.equal(a, b) for a, b in zip(*results))


def test_refusals():
    refs, table, lens = dev([0] * 8), dev([[0] * 4] * 2), dev([0, 0])
    codes, scales = q().new_cache(8, 16, 2, 64)
    keep = torch.zeros(2, dtype=torch.bool, device="cuda")
    for bad in (lambda: q().qcache_reserve(refs, table, lens[:1], 16), lambda: q().qcache_reserve(refs, table, lens, 16, cu=dev([0, 1])),
                lambda: q().qcache_reserve(refs, table, lens, 16, cu=dev([0, 1, 2])), lambda: q().qcache_reserve(refs, table, lens, 16, total=3),
                lambda: q().qcache_reserve(refs, table.T, lens, 16), lambda: q().qcache_fork(refs, table, lens, table, 16),
                lambda: q().qcache_copy(codes, scales, dev([1, 2])), lambda: q().qcache_copy(codes, scales, dev([[1, 2, 3]])),
                lambda: q().qcache_compact(codes, scales, table, lens, keep[:1]), lambda: q().qcache_compact(codes, scales, table, lens, keep, cu_q=dev([0]))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q().qcache_reserve(refs.long(), table, lens, 16), lambda: q().qcache_fork(refs, table, lens, lens.long(), 16),
                lambda: q().qcache_copy(codes, scales, dev([[1, 2]], torch.int64)), lambda: q().qcache_compact(codes, scales, table, lens, keep.int())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: q().qcache_reserve(refs, table, lens, 24), lambda: q().qcache_fork(refs, table, lens, lens, 0)):
        with pytest.raises(q().Qw3Error) as e:
            bad()
        assert e.value.status == q().QW3_ERR_SHAPE


def test_all_holders_of_a_page_take_tokens_in_one_call():
    """Three that share a partly filled page need three pages; with two the last has room in the next call, in the page itself."""
    size, pages = 16, 5
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    table, lens = dev([[-1] * 3]), dev([0])
    _, lens, _ = q().qcache_reserve(refs, table, lens, size, cu=dev([0, 40]), total=40)
    table, lens = q().qcache_fork(refs, table, lens, dev([0, 0, 0]), size)
    assert refs.tolist() == [3, 3, 3, 0, 0]
    slots, lens, copies = q().qcache_reserve(refs, table, lens, size)
    assert slots.tolist() == [3 * 16 + 8, 4 * 16 + 8, -1] and lens.tolist() == [41, 41, 40]
    assert copies.tolist() == [[2, 3], [2, 4], [-1, -1]] and refs.tolist() == [3, 3, 1, 1, 1]
    slots, lens, copies = q().qcache_reserve(refs, table, lens, size)
    assert slots.tolist() == [3 * 16 + 9, 4 * 16 + 9, 2 * 16 + 8] and lens.tolist() == [42, 42, 41]
    assert (copies == -1).all() and table.tolist() == [[0, 1, 3], [0, 1, 4], [0, 1, 2]]
    # with a page for each the old one goes free
    refs = dev([3, 3, 3, 0, 0, 0])
    slots, _, copies = q().qcache_reserve(refs, dev([[0, 1, 2]] * 3), dev([40] * 3), size)
    assert refs.tolist() == [3, 3, 0, 1, 1, 1] and copies.tolist() == [[2, 3], [2, 4], [2, 5]] and (slots % 16 == 8).all()
