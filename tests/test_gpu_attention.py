"""The key/value cache and attention on the GPU against the definitions in 64
bits (oracle/attention.py), through the binding and so through the C ABI.

Codes, scales and values read back are bit-exact.  Attention outputs stay inside
the bound that the oracle derives for each output (attend)."""
import sys

import numpy as np
import pytest
import torch

from oracle import attention as ref

pytestmark = pytest.mark.gpu

TORCH = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def q():
    import dequant_gemv_qgemv_amd as mod
    return mod


def say(*args):
    print("[gpu-case]", *args, file=sys.stderr, flush=True)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def bits(t):
    """bf16 tensor -> uint16 patterns, every NaN the same."""
    u = t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    nan = (u & 0x7FFF) > 0x7F80
    return np.where(nan, np.uint16(0x7FC0), u)


def starts(n):
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")


def rows(rng, n, heads, dim, dtype=torch.bfloat16):
    x = torch.tensor(rng.standard_normal((n, heads, dim)), dtype=torch.float32)
    return x.to(dtype).cuda()


# ------------------------------------------------------------------ cache ---
SPECIAL = {0: "zero", 1: "tiny", 2: "inf", 3: "nan", 4: "huge", 5: "ties", 6: "denormal"}


def special_rows(x, dtype):
    """Rows that quantisation can get wrong, in the first tokens of head 0."""
    d = x.shape[2]
    if x.shape[0] < 8:
        return x
    x[0, 0] = 0.0
    x[1, 0] *= 1e-30
    x[2, 0, d // 2] = float("inf")
    x[3, 0, 1] = float("nan")
    x[4, 0] *= 1e36
    x[5, 0] = (torch.arange(d) % 19 - 9).float().cuda() + 0.5  # with amax 127: exact halves
    x[5, 0, 0] = 127.0
    x[6, 0] = 0.0
    x[6, 0, 3] = 2e-40  # a denormal, also in bf16
    x[7, 0, 0] = -float("inf")
    return x


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("src", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,heads,dim,page", [(1, 1, 64, 16), (9, 3, 128, 16), (70, 2, 64, 64), (33, 8, 128, 32)])
def test_write_is_exact(kind, src, tokens, heads, dim, page):
    say("write", kind, src, tokens, heads, dim, page)
    rng = np.random.default_rng(tokens + dim)
    pages = -(-tokens // page) + 2
    codes, scales = q().new_cache(pages, page, heads, dim, TORCH[kind])
    codes.view(torch.uint8).fill_(0x5A)
    scales.fill_(-7.0)
    # views of one fused projection output: [q | k | v] per token
    fused = torch.zeros(tokens, (2 * heads + 5) * dim, dtype=src, device="cuda")
    k = fused[:, 2 * dim:(2 + heads) * dim].view(tokens, heads, dim)
    v = fused[:, (3 + heads) * dim:(3 + 2 * heads) * dim].view(tokens, heads, dim)
    k.copy_(special_rows(rows(rng, tokens, heads, dim, src), src))
    v.copy_(rows(rng, tokens, heads, dim, src))
    slots = torch.tensor(rng.permutation(pages * page)[:tokens], dtype=torch.int64)
    if tokens > 8:
        slots[8] = -1                 # padding
    if tokens > 30:
        slots[9] = pages * page       # out of range: stores nothing
        slots[10] = 2 ** 40
    q().qcache_write(k, v, slots.cuda(), codes, scales)
    want_c = np.full((pages, 2, heads, page, dim), 0x5A, np.uint8)
    want_s = np.full((pages, 2, heads, page), -7.0, np.float32)
    for which, x in enumerate((k, v)):
        c, s = ref.quantise(x.float().cpu().numpy(), kind)
        for t, slot in enumerate(slots.tolist()):
            if 0 <= slot < pages * page:
                want_c[slot // page, which, :, slot % page] = c[t]
                want_s[slot // page, which, :, slot % page] = s[t]
    got_c, got_s = codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy()
    assert np.array_equal(got_s, want_s, equal_nan=True)
    if kind == "e4m3":  # a negative zero is a zero
        got_c, want_c = np.where(got_c == 0x80, 0, got_c), np.where(want_c == 0x80, 0, want_c)
    assert np.array_equal(got_c, want_c)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_quotients_at_rounding_boundaries(kind):
    """Elements within a few floats of a boundary between two codes, for many scales, tiny and huge ones among them:
    codes are those of the correctly rounded quotient."""
    rng = np.random.default_rng(23)
    tokens, heads, dim = 600, 1, 128
    limit = np.float32(ref.LIMIT[kind])
    if kind == "int8":
        middle = rng.integers(-127, 127, (tokens, heads, dim)) + 0.5
    else:
        v = ref.e4m3_table()[:127]
        at = rng.integers(0, 126, (tokens, heads, dim))
        middle = (v[at] + v[at + 1]) / 2 * rng.choice([-1, 1], at.shape)
    top = (limit * np.exp2(rng.integers(-100, 100, (tokens, heads, 1))) * rng.uniform(0.6, 1.9, (tokens, heads, 1))).astype(np.float32)
    scale = top / limit
    x = (middle * scale).astype(np.float32)
    for _ in range(3):
        x = np.nextafter(x, np.where(rng.random(x.shape) < 0.5, -np.inf, np.inf).astype(np.float32))
    x[:, :, 0] = top[:, :, 0]
    codes, scales = q().new_cache(tokens // 16 + 1, 16, heads, dim, TORCH[kind])
    k = torch.tensor(x).cuda()
    q().qcache_write(k, k, torch.arange(tokens, device="cuda"), codes, scales)
    want_c, want_s = ref.quantise(x, kind)
    got = codes.view(torch.uint8).cpu().numpy()[:, 0].transpose(0, 2, 1, 3).reshape(-1, heads, dim)[:tokens]
    got_s = scales.cpu().numpy()[:, 0].transpose(0, 2, 1).reshape(-1, heads)[:tokens]
    if kind == "e4m3":
        got, want_c = np.where(got == 0x80, 0, got), np.where(want_c == 0x80, 0, want_c)
    assert np.array_equal(got_s, want_s) and np.array_equal(got, want_c)


def random_cache(rng, kind, pages, page, heads, dim):
    raw = torch.tensor(rng.integers(0, 256, (pages, 2, heads, page, dim)), dtype=torch.uint8)
    if kind == "int8":
        raw[raw == 0x80] = 0x81  # -128 is not written
    else:
        raw[(raw & 0x7F) == 0x7F] = 0x3C
    scales = torch.tensor(np.exp(rng.standard_normal((pages, 2, heads, page))) * (0.02 if kind == "int8" else 0.005),
                          dtype=torch.float32)
    return raw.cuda().view(TORCH[kind]), scales.cuda()


def tables(rng, lens, page, pages, spare=1):
    """A block table over distinct random pages; entries past a sequence's end are out of range."""
    need = [-(-n // page) for n in lens]
    ids = rng.permutation(pages)
    t = np.full((len(lens), max(need + [0]) + spare), 2 ** 31 - 1, np.int32)
    at = 0
    for b, c in enumerate(need):
        t[b, :c] = ids[at:at + c]
        at += c
    return torch.tensor(t, device="cuda")


@pytest.mark.parametrize("kind,heads,dim,page,lens", [
    ("int8", 1, 64, 16, [1]), ("int8", 8, 128, 16, [0, 17, 0, 1, 130, 15]), ("e4m3", 3, 128, 64, [63, 64, 65]),
    ("e4m3", 5, 64, 32, [33] * 70), ("int8", 2, 128, 128, [500, 3]),
    ("int8", 3, 64, 32, [9001, 5, 7500])])
def test_read_is_exact(kind, heads, dim, page, lens):
    say("read", kind, heads, dim, page, lens[:8])
    rng = np.random.default_rng(len(lens))
    pages = sum(-(-n // page) for n in lens) + 3
    codes, scales = random_cache(rng, kind, pages, page, heads, dim)
    scales[0, 0, 0, 0] = float("nan")
    table = tables(rng, lens, page, pages)
    total = sum(lens) + 5  # rows of no sequence stay as they are
    out = [torch.full((total, heads, dim), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q().qcache_read(codes, scales, table, starts(lens), total, out=out)
    c = codes.view(torch.uint8).cpu().numpy()
    val = ref.code_values(c, kind).astype(np.float32) * scales.cpu().numpy()[..., None]
    tab = table.cpu().numpy()
    for which in (0, 1):
        got, at = bits(out[which]), 0
        for b, n in enumerate(lens):
            want = np.concatenate([val[p, which].transpose(1, 0, 2) for p in tab[b, :-(-n // page)]] or [val[0, 0, :, :0].transpose(1, 0, 2)])[:n]
            assert np.array_equal(got[at:at + n], ref.to_bf16(want)), (which, b)
            at += n
        assert (got[at:] == 0x4110).all()


def test_read_of_pages_that_do_not_exist_gives_zeros():
    rng = np.random.default_rng(5)
    codes, scales = random_cache(rng, "int8", 4, 16, 2, 64)
    table = torch.tensor([[1, -1, 4], [2 ** 31 - 1, 0, -(2 ** 31)]], dtype=torch.int32, device="cuda")
    k, v = q().qcache_read(codes, scales, table, starts([60, 48]), 108)  # 60 tokens: 12 past the table
    for t in (k, v):
        t = f64(t)
        assert np.abs(t[:16]).sum() > 0 and np.abs(t[60 + 16:60 + 32]).sum() > 0
        assert (t[16:60] == 0).all() and (t[60:76] == 0).all() and (t[92:] == 0).all()


def check(got, want, bound, what):
    err = np.abs(got - want)
    bad = ~(err <= bound)
    bad &= ~(np.isnan(got) & np.isnan(want))
    assert not bad.any(), "%s: %d outputs off, the worst %g times the bound" % (
        what, bad.sum(), np.nanmax(np.where(bad, err / np.maximum(bound, 1e-300), 0)))


def cache_case(rng, kind, heads, group, dim, page, lens, news, tree, scale=None, touch=None, pages=None, some=None):
    """One qattn_cache call against the oracle, every row and head (`some`: that many rows of each sequence).
    With many rows a second one, whose table is wide enough for the kernels of large calls."""
    news = [news] * len(lens) if isinstance(news, int) else news
    pages = pages or sum(-(-n // page) for n in lens) + 2
    codes, scales = random_cache(rng, kind, pages, page, heads, dim)
    table = tables(rng, lens, page, pages)
    rq = rows(rng, sum(news), heads * group, dim)
    words = None
    if tree:
        words = torch.tensor(rng.integers(-2 ** 63, 2 ** 63, sum(news)), dtype=torch.int64)
        if len(words) > 2:
            words[1] = 0   # a row that sees no draft
            words[2] = -1
    if touch:
        touch(codes, scales, table, rq, words)
    kw = {} if scale is None else dict(sm_scale=scale)
    if not all(n == 1 for n in news):
        kw["cu_q"] = starts(news)
    out = torch.full(rq.shape, 77.0, dtype=torch.bfloat16, device="cuda")
    q().qattn_cache(rq, codes, scales, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                    tree=words.cuda() if words is not None else None, out=out, **kw)
    outs, qq = [f64(out)], f64(rq)
    if -(-sum(news) // len(lens)) * group > 64:
        width = (1 << 25) // (page * rq.shape[0] * rq.shape[1]) + 1
        wide = torch.full((len(lens), max(width, table.shape[1])), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = table
        out.fill_(77.0)
        q().qattn_cache(rq, codes, scales, wide, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                        tree=words.cuda() if words is not None else None, out=out, **kw)
        outs.append(f64(out))
    val = ref.code_values(codes.view(torch.uint8).cpu().numpy(), kind) * scales.cpu().numpy().astype(np.float64)[..., None]
    tab, at = table.cpu().numpy(), 0
    for b, (n, length) in enumerate(zip(news, lens)):
        tokens = np.arange(length)
        page_of = tab[b, tokens // page] if length else np.zeros(0, int)
        there = (page_of >= 0) & (page_of < pages)
        kv = val[np.where(there, page_of, 0), :, :, tokens % page]  # [len, 2, H, D]
        for i in range(n) if some is None or n <= some else sorted(rng.choice(n, some, replace=False).tolist()):
            sees = ref.cache_sees(i, n, length, int(words[at + i]) & (2 ** 64 - 1) if tree else None)
            sees = sees[there[sees]] if len(sees) else sees
            for h in range(heads * group):
                o, bound = ref.attend(qq[at + i, h], kv[:, 0, h // group], kv[:, 1, h // group], sees,
                                      dim ** -0.5 if scale is None else scale)
                for got in outs:
                    check(got[at + i, h], o, bound, "sequence %d row %d head %d" % (b, i, h))
        at += n


@pytest.mark.parametrize("kind,dim", [("int8", 128), ("e4m3", 128), ("int8", 64), ("e4m3", 64)])
@pytest.mark.parametrize("heads,group,page,lens", [
    (1, 1, 16, [1]), (2, 8, 16, [15, 16, 17, 31, 33]), (1, 5, 32, [127, 128, 129, 0, 255]), (3, 4, 64, [1000, 1, 513]),
    (2, 7, 128, [300])])
def test_single_tokens(kind, dim, heads, group, page, lens):
    say("single", kind, dim, heads, group, page, lens)
    cache_case(np.random.default_rng(heads * 100 + group), kind, heads, group, dim, page, lens, 1, False)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("kind,heads,group,dim,page,lens,news", [
    ("int8", 2, 8, 128, 16, [70, 40, 300], [2, 3, 1]),      # 16-row blocks, odd rows
    ("e4m3", 1, 4, 64, 32, [200, 8], 8),                     # 32 rows
    ("int8", 1, 8, 128, 16, [90, 64], [64, 33]),             # 64-row blocks, several per sequence
    ("e4m3", 2, 3, 128, 64, [129, 40, 31], [31, 0, 31]),     # a sequence with no new token, one with no context
    ("int8", 1, 1, 64, 16, [7, 5, 0, 100], [7, 9, 2, 70]),   # more new tokens than cached ones; more than 64
    ("e4m3", 1, 8, 64, 32, [100, 65, 17], [30, 9, 17]),      # 128-row blocks, e4m3 codes
    ("e4m3", 2, 5, 128, 16, [63, 200, 1], [40, 13, 1]),
])
def test_drafts(tree, kind, heads, group, dim, page, lens, news):
    say("drafts", tree, kind, heads, group, dim, page, lens, news)
    cache_case(np.random.default_rng(sum(lens)), kind, heads, group, dim, page, lens, news, tree)


def test_many_sequences():
    """More sequences than lanes, many of them empty; two rows for some."""
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 40, 150)]
    news = [int(x) for x in rng.integers(0, 3, 150)]
    cache_case(rng, "int8", 2, 2, 64, 16, lens, news, False)


def test_a_long_sequence_beside_short_ones():
    cache_case(np.random.default_rng(4), "int8", 1, 8, 128, 16, [20000, 3, 700], 1, False)
    cache_case(np.random.default_rng(5), "e4m3", 2, 2, 64, 64, [9000, 70], [3, 5], True)
    cache_case(np.random.default_rng(55), "int8", 1, 24, 64, 32, [7000, 40, 900], [4, 3, 4], True)


@pytest.mark.parametrize("kind,group,dim,length,news", [
    ("int8", 8, 128, 9000, 1), ("e4m3", 5, 64, 5003, 4), ("int8", 2, 128, 2500, 50), ("e4m3", 4, 128, 2100, 40)])
def test_long_sequences_of_one_head(kind, group, dim, length, news):
    """Fewer workgroups than the card has: the runs are cut for the longest item's join."""
    cache_case(np.random.default_rng(21), kind, 1, group, dim, 16, [length, 3 + news], news, news > 1)


@pytest.mark.parametrize("kind,lens", [("int8", [300, 1100]), ("e4m3", [64, 777])])
def test_more_rows_than_the_card_has_workgroups(kind, lens):
    cache_case(np.random.default_rng(25), kind, 2, 128, 128, 16, lens, 64, True, some=5)


def test_many_rows_of_many_sequences():
    """128-row blocks: items that share a workgroup, and items that several share."""
    rng = np.random.default_rng(56)
    lens = [int(x) for x in rng.integers(0, 90, 70)]
    cache_case(rng, "int8", 1, 33, 64, 16, lens, [int(x) for x in rng.integers(1, 4, 70)], False)


@pytest.mark.parametrize("scale", [0.01, 1.0, 40.0])
def test_other_scales(scale):
    """A flat softmax, and one that a single key decides."""
    cache_case(np.random.default_rng(6), "int8", 2, 4, 128, 16, [200, 37], 2, True, scale=scale)


@pytest.mark.parametrize("group", [4, 20])
def test_what_is_hidden_has_no_influence(group):
    """NaN scales of hidden drafts, garbage past the end (codes that are NaN in e4m3 too) and missing pages."""
    def touch(codes, scales, table, rq, words):
        raw = codes.view(torch.uint8)
        # sequence 0 has 50 tokens on pages of 16: the rest of its last page is garbage
        last = int(table[0, 3])
        raw[last, :, :, 2:] = 0x7F
        scales[last, :, :, 2:] = float("nan")
        # draft 2 of sequence 1 (tokens 36..39): NaN; only rows whose word has bit 2 see it
        p = int(table[1, 2])
        scales[p, :, :, 38 % 16] = float("nan")
        for i in range(4):
            words[4 + i] = (1 << i) | (4 if i == 3 else 0)
        # the second page of sequence 2 does not exist
        table[2, 1] = -5

    for kind in ("int8", "e4m3"):
        cache_case(np.random.default_rng(7), kind, 2, group, 128, 16, [50, 40, 60], 4, True, touch=touch)


@pytest.mark.parametrize("group", [2, 66])
def test_nan_and_zero_rows_that_are_seen(group):
    def touch(codes, scales, table, rq, words):
        scales[int(table[0, 0]), 0, 0, 3] = float("nan")   # a key of head 0
        scales[int(table[1, 0]), 1, 1, 3] = float("nan")   # a value of head 1
        scales[int(table[2, 0])] = 0.0                     # rows of zeros

    cache_case(np.random.default_rng(8), "int8", 2, group, 64, 16, [20, 20, 16], 1, False, touch=touch)


@pytest.mark.parametrize("group", [8, 66])
def test_scales_of_very_different_sizes(group):
    """Value scales over 2^40: each weight is rounded relative to itself."""
    def touch(codes, scales, table, rq, words):
        e = torch.tensor(np.random.default_rng(1).integers(-20, 20, tuple(scales[:, 1].shape)), device="cuda")
        scales[:, 1] = torch.exp2(e.float())

    cache_case(np.random.default_rng(9), "int8", 1, group, 128, 16, [333], 1, False, touch=touch)


def test_cache_beyond_4_gib():
    """Pages whose codes start past 2^32 bytes, written, read back and attended to."""
    rng = np.random.default_rng(10)
    heads, dim, page, n = 8, 128, 16, 100
    pages = (1 << 32) // (2 * heads * page * dim) + 40
    codes = torch.empty(pages, 2, heads, page, dim, dtype=torch.int8, device="cuda")
    scales = torch.empty(pages, 2, heads, page, dtype=torch.float32, device="cuda")
    table = torch.arange(pages - 20, pages - 13, dtype=torch.int32, device="cuda").view(1, -1)
    k, v = rows(rng, n, heads, dim), rows(rng, n, heads, dim)
    slots = (pages - 20) * page + torch.arange(n, device="cuda")
    q().qcache_write(k, v, slots, codes, scales)
    kr, vr = q().qcache_read(codes, scales, table, starts([n]), n)
    for x, back in ((k, kr), (v, vr)):
        c, s = ref.quantise(x.float().cpu().numpy(), "int8")
        assert np.array_equal(bits(back), ref.to_bf16(c.view(np.int8).astype(np.float32) * s[..., None]))
    rq = rows(rng, 1, 64, dim)
    got = f64(q().qattn_cache(rq, codes, scales, table, torch.tensor([n], dtype=torch.int32, device="cuda")))
    c, s = ref.quantise(np.stack([k.float().cpu().numpy(), v.float().cpu().numpy()]), "int8")
    val = c.view(np.int8).astype(np.float64) * s[..., None]
    for h in range(64):
        o, bound = ref.attend(f64(rq)[0, h], val[0][:, h // 8], val[1][:, h // 8], np.arange(n), dim ** -0.5)
        check(got[0, h], o, bound, "head %d" % h)


# ----------------------------------------------------------------- prompt ---
def prompt_case(rng, nq, nk, heads, group, dim, causal, scale=None, touch=None, some=None, fused=False):
    """One qattn_prompt call against the oracle; `some`: how many rows of each sequence are checked (all)."""
    tq, tk = sum(nq), sum(nk)
    rq = rows(rng, tq, heads * group, dim)
    if fused:  # k and v as views of one [tokens, (k | v) per head, 2 D] tensor, head stride 2 D
        kv = rows(rng, tk, heads, 2 * dim)
        rk, rv = kv[:, :, :dim], kv[:, :, dim:]
        wide = torch.zeros(tq, heads * group + 3, dim, dtype=torch.bfloat16, device="cuda")
        wide[:, 1:1 + heads * group] = rq
        rq = wide[:, 1:1 + heads * group]
    else:
        rk, rv = rows(rng, tk, heads, dim), rows(rng, tk, heads, dim)
    if touch:
        touch(rq, rk, rv)
    kw = {} if scale is None else dict(sm_scale=scale)
    out = torch.full((tq + 3, heads * group, dim), 77.0, dtype=torch.bfloat16, device="cuda")
    q().qattn_prompt(rq, rk, rv, starts(nq), None if nq == nk else starts(nk), causal=causal, out=out[:tq], **kw)
    got, qq, kk, vv = f64(out), f64(rq), f64(rk), f64(rv)
    assert (got[tq:] == 77).all()
    q0 = k0 = 0
    for b, (a, c) in enumerate(zip(nq, nk)):
        pick = range(a) if some is None or a <= some else sorted({0, a - 1} | set(rng.integers(0, a, some).tolist()))
        for i in pick:
            sees = ref.prompt_sees(i, a, c, causal)
            for h in range(heads * group):
                o, bound = ref.attend(qq[q0 + i, h], kk[k0:k0 + c, h // group], vv[k0:k0 + c, h // group], sees,
                                      dim ** -0.5 if scale is None else scale)
                check(got[q0 + i, h], o, bound, "sequence %d row %d head %d" % (b, i, h))
        q0, k0 = q0 + a, k0 + c


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nq,heads,group", [
    ([1], 1, 1), ([37], 2, 8), ([63, 64, 65, 1, 2], 1, 3), ([127, 0, 128, 129], 2, 1), ([300, 31, 33], 1, 5)])
def test_prompts(causal, dim, nq, heads, group):
    say("prompt", causal, dim, nq, heads, group)
    prompt_case(np.random.default_rng(sum(nq)), nq, nq, heads, group, dim, causal, some=40)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nq,nk", [
    ([1], [5000]), ([20, 130], [500, 131]), ([64, 3, 40], [0, 3, 10]), ([200], [70])])
def test_chunks(causal, dim, nq, nk):
    """More keys than queries (a chunk of a prompt), fewer (rows that see nothing), none at all."""
    say("chunk", causal, dim, nq, nk)
    prompt_case(np.random.default_rng(sum(nk)), nq, nk, 2, 2, dim, causal, some=40)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim,nq,nk,heads,group", [
    (128, [1], [4000], 1, 1), (64, [33, 2, 70], [1500, 0, 700], 1, 3), (128, [65], [2049], 2, 2),
    (64, [64, 1], [129, 6000], 1, 1), (128, [90], [150], 1, 4)])
def test_few_rows_against_many_keys(causal, dim, nq, nk, heads, group):
    """The keys of a tile in slices: of one tile, of unequal length, past a row's last key."""
    say("slices", causal, dim, nq, nk)
    prompt_case(np.random.default_rng(sum(nk) + 1), nq, nk, heads, group, dim, causal, some=12)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nonfinite_values_in_slices(dim, bad):
    """A key in the middle that all rows see (one channel), the last ones that some see."""
    rng = np.random.default_rng(22)
    rq, rk, rv = rows(rng, 40, 2, dim), rows(rng, 1500, 1, dim), rows(rng, 1500, 1, dim)
    rv[1490, 0, :] = bad
    cu, cuk = starts([40]), starts([1500])
    got = f64(q().qattn_prompt(rq, rk, rv, cu, cuk))
    for i in (0, 13, 29):  # row i sees the keys up to 1460 + i
        for h in (0, 1):
            o, bound = ref.attend(f64(rq)[i, h], f64(rk)[:, 0], f64(rv)[:, 0], np.arange(1461 + i), dim ** -0.5)
            check(got[i, h], o, bound, "row %d head %d" % (i, h))
    assert not np.isfinite(got[30:]).any()
    rv[700, 0, 5] = bad
    again = f64(q().qattn_prompt(rq, rk, rv, cu, cuk))
    assert not np.isfinite(again[:, :, 5]).any()
    assert np.isfinite(np.delete(again[:30], 5, axis=2)).all()


def test_many_prompts():
    rng = np.random.default_rng(11)
    nq = [int(x) for x in rng.integers(0, 30, 140)]
    prompt_case(rng, nq, nq, 1, 2, 64, True, some=2)


def test_longer_prompts():
    rng = np.random.default_rng(12)
    prompt_case(rng, [1500, 700], [1500, 700], 2, 4, 128, True, some=6)
    prompt_case(rng, [2049], [2049], 1, 2, 64, False, some=6)


def test_strided_views():
    prompt_case(np.random.default_rng(13), [150, 20], [150, 20], 2, 3, 128, True, fused=True, some=30)
    prompt_case(np.random.default_rng(14), [70], [90], 1, 2, 64, False, fused=True)


@pytest.mark.parametrize("scale", [0.003, 1.0, 30.0])
def test_prompt_scales(scale):
    prompt_case(np.random.default_rng(15), [100], [100], 1, 2, 128, True, scale=scale)


def test_growing_scores():
    """Keys whose scores grow along the sequence, so that the running maximum moves in every tile."""
    def touch(rq, rk, rv):
        rk.copy_(rq[:, :1] * torch.linspace(0.1, 6, rk.shape[0], device="cuda").view(-1, 1, 1).bfloat16())
        rq.copy_(rq[:1].expand_as(rq).clone())

    prompt_case(np.random.default_rng(16), [400], [400], 1, 1, 128, True, touch=touch, some=50)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_nonfinite_values_reach_only_rows_that_see_them(dim, bad):
    """Of a later token, and of the sequence behind: keys and values."""
    def touch(rq, rk, rv):
        rv[90, 0, 5] = bad
        rk[100, 0, 7] = bad
        rv[130, 0, :] = bad

    rng = np.random.default_rng(17)
    tq = [120, 40]
    rq, rk, rv = rows(rng, 160, 2, dim), rows(rng, 160, 1, dim), rows(rng, 160, 1, dim)
    clean = q().qattn_prompt(rq, rk, rv, starts(tq))
    touch(rq, rk, rv)
    got = q().qattn_prompt(rq, rk, rv, starts(tq))
    for i in (0, 50, 89, 120, 129):  # see nothing of it
        for h in (0, 1):
            base = 0 if i < 120 else 120
            o, bound = ref.attend(f64(rq)[i, h], f64(rk)[base:, 0], f64(rv)[base:, 0], np.arange(i - base + 1), dim ** -0.5)
            check(f64(got)[i, h], o, bound, "row %d head %d" % (i, h))
            check(f64(clean)[i, h], o, bound, "row %d head %d" % (i, h))
    g = f64(got)
    assert not np.isfinite(g[90:100, :, 5]).any()
    assert np.isfinite(np.delete(g[90:100], 5, axis=2)).all()
    assert not np.isfinite(g[130:]).any()


# ------------------------------------------------------------ the machine ---
def layer_inputs(rng, kind="int8"):
    lens = [333, 4000, 20]
    codes, scales = random_cache(rng, kind, 300, 16, 8, 128)
    return dict(codes=codes, scales=scales, block_table=tables(rng, lens, 16, 300),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def test_deterministic():
    rng = np.random.default_rng(18)
    c = layer_inputs(rng)
    rq = rows(rng, 12, 64, 128)
    cu = starts([4, 5, 3])
    first = bits(q().qattn_cache(rq, cu_q=cu, **c))
    p = rows(rng, 700, 8, 128)
    pk = rows(rng, 700, 2, 128)
    second = bits(q().qattn_prompt(p, pk, pk, starts([300, 400])))
    for _ in range(3):
        assert np.array_equal(first, bits(q().qattn_cache(rq, cu_q=cu, **c)))
        assert np.array_equal(second, bits(q().qattn_prompt(p, pk, pk, starts([300, 400]))))


def test_streams_and_graph_replay():
    """A decode step captured on a stream of its own: write, attend, read back; every replay against eager calls."""
    rng = np.random.default_rng(19)
    c = layer_inputs(rng)
    k, v, rq = rows(rng, 3, 8, 128), rows(rng, 3, 8, 128), rows(rng, 3, 64, 128)
    slots = c["block_table"].long().gather(1, ((c["lens"].long() - 1) // 16)[:, None])[:, 0] * 16 + (c["lens"].long() - 1) % 16
    p, pk = rows(rng, 200, 8, 128), rows(rng, 200, 2, 128)
    cu, cur = starts([150, 50]), starts([333, 4000, 20])

    def step():
        q().qcache_write(k, v, slots, c["codes"], c["scales"])
        return (q().qattn_cache(rq, **c), *q().qcache_read(c["codes"], c["scales"], c["block_table"], cur, 4353),
                q().qattn_prompt(p, pk, pk, cu))

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = step()
    for _ in range(4):
        for t in (k, v, rq, p, pk):
            t.copy_(rows(rng, *t.shape))
        graph.replay()
        torch.cuda.synchronize()
        got = [bits(t) for t in outs]
        want = [bits(t) for t in step()]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert np.array_equal(a, b)


def test_slices_repeat_and_replay():
    """Parts joined by whoever finishes last: the same bits every time, eager and in a graph."""
    rng = np.random.default_rng(23)
    rq, rk, rv = rows(rng, 70, 4, 128), rows(rng, 5000, 1, 128), rows(rng, 5000, 1, 128)
    cu, cuk = starts([50, 20]), starts([1800, 3200])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        first = bits(q().qattn_prompt(rq, rk, rv, cu, cuk))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = q().qattn_prompt(rq, rk, rv, cu, cuk)
    for _ in range(4):
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits(out), first)
        assert np.array_equal(bits(q().qattn_prompt(rq, rk, rv, cu, cuk)), first)


def test_two_streams_at_once():
    """Each stream has a workspace of its own."""
    rng = np.random.default_rng(20)
    c = layer_inputs(rng)
    qs = [rows(rng, 3, 64, 128) for _ in range(6)]
    want = [bits(q().qattn_cache(x, **c)) for x in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i, x in enumerate(qs):
        with torch.cuda.stream(streams[i % 2]):
            got.append(q().qattn_cache(x, **c))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert np.array_equal(bits(a), b)


def test_a_product_between_two_attention_calls():
    """The products and attention share a stream's workspace: neither leaves anything in it that the other needs."""
    rng = np.random.default_rng(21)
    c = layer_inputs(rng)
    rq = rows(rng, 3, 64, 128)
    want = bits(q().qattn_cache(rq, **c))
    packed = q().qpack_uint3(torch.tensor(rng.integers(0, 8, (512, 1024)), dtype=torch.uint8, device="cuda"))
    s = torch.full((512, 8), 0.01, dtype=torch.bfloat16, device="cuda")
    x = rows(rng, 40, 1, 1024)[:, 0].contiguous()
    y = q().qgemm_w3g128_smallM(x, packed, s)
    for _ in range(3):
        assert np.array_equal(want, bits(q().qattn_cache(rq, **c)))
        assert torch.equal(y, q().qgemm_w3g128_smallM(x, packed, s))


@pytest.mark.parametrize("rows_per_head", [1, 40])
def test_starts_and_lengths_out_of_range_are_clipped(rows_per_head):
    """Starts past the rows, decreasing or negative; lengths past the table: nothing outside the arrays is touched."""
    rng = np.random.default_rng(24)
    codes, scales = random_cache(rng, "int8", 8, 16, 2, 64)
    table = tables(rng, [30, 40, 20], 16, 8)
    heads = 2 * rows_per_head
    rq = rows(rng, 9, heads, 64)
    wide = torch.full((3, (1 << 24) // (16 * 9 * heads) + 1), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table  # with many rows: the kernel of large calls
    guard = torch.full((9 + 4, heads, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    for cu in ([0, 2000, 4, 9], [-7, 3, 3, 1 << 30], [5, 2, 9, 9]):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        lens = torch.tensor([30, 1 << 30, -4], dtype=torch.int32, device="cuda")
        for t in (table, wide):
            q().qattn_cache(rq, codes, scales, t, lens, cu_q=c, out=guard[:9])
        k = rows(rng, 9, 2, 64)
        q().qattn_prompt(rq, k, k, c, out=guard[:9])
        q().qattn_prompt(rq, k, k, c, causal=False, out=guard[:9])
        out = [torch.full((13, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        q().qcache_read(codes, scales, table, c, 9, out=[t[:9] for t in out])
        torch.cuda.synchronize()
        assert (guard[9:] == 5).all() and all((t[9:] == 5).all() for t in out)


@pytest.mark.parametrize("codes", [torch.int8, torch.float8_e4m3fn])
def test_example(codes):
    """The four calls together, as a server uses them: prompts in chunks, a drafted tree, the accepted path."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")
    spec = importlib.util.spec_from_file_location("attention_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    # 8-bit keys and values: int8 rounds by up to 1/254 of a row's largest element, e4m3 an element by up to 1/16
    assert mod.demo(codes=codes, verbose=False) < (0.02 if codes is torch.int8 else 0.08)


def test_refusals_on_the_gpu():
    rng = np.random.default_rng(22)
    c = layer_inputs(rng)
    rq = rows(rng, 3, 64, 128)
    with pytest.raises(ValueError):
        q().qattn_cache(rq[:2], **c)                      # one row per sequence without cu_q
    with pytest.raises(ValueError):
        q().qattn_cache(rq[:, :60].contiguous(), **c)     # 60 heads over 8
    with pytest.raises(TypeError):
        q().qattn_cache(rq.float(), **c)
    with pytest.raises(ValueError):
        q().qattn_cache(rq, **{**c, "scales": c["scales"][:4]})
    with pytest.raises(TypeError):
        q().qattn_cache(rq, tree=torch.zeros(3, dtype=torch.int32, device="cuda"), **c)
    with pytest.raises(ValueError):
        q().qattn_cache(rq.transpose(1, 2).contiguous().transpose(1, 2), **c)  # channels not contiguous
    with pytest.raises(q().Qw3Error) as e:
        q().qattn_cache(rq, sm_scale=-1.0, **c)
    assert e.value.status == q().QW3_ERR_SHAPE
    with pytest.raises(q().Qw3Error) as e:
        x = torch.zeros(3 * 64 * 128 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(3, 64, 128)
        q().qattn_cache(x, **c)
    assert e.value.status == q().QW3_ERR_ALIGN
    k = rows(rng, 3, 8, 128)
    with pytest.raises(ValueError):
        q().qcache_write(k, k, torch.zeros(2, dtype=torch.int64, device="cuda"), c["codes"], c["scales"])
    with pytest.raises(TypeError):
        q().qcache_write(k, k.float(), torch.zeros(3, dtype=torch.int64, device="cuda"), c["codes"], c["scales"])
    with pytest.raises(ValueError):
        q().qcache_write(k[:, :4], k[:, :4], torch.zeros(3, dtype=torch.int64, device="cuda"), c["codes"], c["scales"])
    with pytest.raises(ValueError):
        q().qattn_prompt(rq, k, k, starts([3]), starts([1, 2]))
    with pytest.raises(ValueError):
        q().qattn_prompt(rq, k[:, :3], k[:, :3], starts([3]))
    with pytest.raises(ValueError):
        q().qattn_prompt(rq, k, k, starts([3]), out=torch.empty(3, 64, 64, dtype=torch.bfloat16, device="cuda"))
