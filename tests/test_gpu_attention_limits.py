"""What the cache and attention calls do at the edges of their arguments: starts,
lengths, codes and values that a server's program should not produce but may."""
import sys

import numpy as np
import pytest
import torch

from oracle import attention as ref
from test_gpu_attention import bits, cache_case, check, f64, q, random_cache, rows, say, starts, tables

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ----------------------------------------------------------------- starts ---
@pytest.mark.parametrize("rows_per_head,dim", [(1, 128), (3, 64), (40, 128)])
def test_starts_that_overlap_leave_later_calls_alone(rows_per_head, dim):
    """A call whose starts name every row many times, more work than 31 bits if counted as it stands; then a valid call
    on the same stream, whose parts several workgroups join, gives its earlier bits, again and again."""
    say("overlapping starts", rows_per_head, dim)
    rng = np.random.default_rng(31)
    lens = [9000, 3000, 17]
    codes, scales = random_cache(rng, "int8", 800, 16, 2, dim)
    table = tables(rng, lens, 16, 800)
    good = rows(rng, 6, 2 * rows_per_head, dim)
    cu = starts([3, 2, 1])
    want = bits(q().qattn_cache(good, codes, scales, table, ints(lens), cu_q=cu))
    n = 3000
    many = rows(rng, n, 2 * rows_per_head, dim)
    jumps = np.zeros(n + 1, np.int32)
    jumps[1::2] = n
    wide = torch.full((n, 64), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    wide[:] = table[0, :64]
    out = torch.full((n + 3, 2 * rows_per_head, dim), 5.0, dtype=torch.bfloat16, device="cuda")
    q().qattn_cache(many, codes, scales, wide, ints([1000] * n), cu_q=ints(jumps), out=out[:n])
    # the starts as they then stand: all rows are the first sequence's
    same = q().qattn_cache(many, codes, scales, wide, ints([1000] * n), cu_q=ints(np.maximum.accumulate(jumps)))
    assert (f64(out[n:]) == 5).all() and np.array_equal(bits(out[:n]), bits(same))
    for _ in range(3):
        assert np.array_equal(want, bits(q().qattn_cache(good, codes, scales, table, ints(lens), cu_q=cu)))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("pad", [0, 70])
def test_falling_starts_of_prompts(causal, pad):
    """A start below an earlier one counts as that one: the outputs are those of the starts as they then stand, and rows
    of no sequence are not written. `pad`: more sequences than a wave has lanes."""
    rng = np.random.default_rng(32)
    rq, rk, rv = rows(rng, 700, 4, 128), rows(rng, 700, 2, 128), rows(rng, 700, 2, 128)
    for cu in ([500, 600, 0, 300, 700], [0, 200, 100, 650, 650], [300, 20, 10, 400, 350], [-5, 1 << 30, 4, 9, 2]):
        cu = cu + [cu[-1]] * pad
        fixed = np.maximum.accumulate(np.clip(cu, 0, 700))
        outs = []
        for c in (cu, fixed):
            out = torch.full((700, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
            q().qattn_prompt(rq, rk, rv, ints(c), ints(fixed), causal=causal, out=out)
            outs.append(bits(out))
        assert np.array_equal(*outs), cu
        assert (outs[0][:max(fixed[0], 0)] == 0x40A0).all() and (outs[0][fixed[-1]:] == 0x40A0).all()


def test_falling_starts_of_reads_and_decodes():
    rng = np.random.default_rng(33)
    codes, scales = random_cache(rng, "int8", 40, 16, 2, 64)
    table = tables(rng, [100, 90, 60, 120], 16, 40)
    rq = rows(rng, 120, 4, 64)
    for cu in ([50, 60, 0, 30, 90], [0, 70, 20, 65, 65], [30, 2, 1, 40, 35], [-5, 1 << 30, 4, 9, 2]):
        fixed = np.maximum.accumulate(np.clip(cu, 0, 120))
        reads, decodes = [], []
        for c in (cu, fixed):
            out = [torch.full((120, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            if c is fixed or cu[0] >= 0:
                q().qcache_read(codes, scales, table, ints(c), 120, out=out)
                reads.append([bits(t) for t in out])
            o = torch.full((120, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
            q().qattn_cache(rq, codes, scales, table, ints([100, 90, 60, 120]), cu_q=ints(c), out=o)
            decodes.append(bits(o))
        assert np.array_equal(*decodes), cu
        if len(reads) == 2:
            assert np.array_equal(*reads), cu


# ------------------------------------------------- codes that are NaN (e4m3) ---
def plant(codes, table, seq, token, which, head, channels, code):
    size = codes.shape[3]
    codes.view(torch.uint8)[int(table[seq, token // size]), which, head, token % size, channels] = code


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [2, 4, 20])
def test_nan_codes_reach_only_rows_that_see_them(group, dim, tree):
    """Places of drafts that were never written, or hold another writer's NaN: values and keys, seen by some rows of a
    block and hidden from others; behind them a context that all rows see and what lies past the end."""
    def touch(codes, scales, table, rq, words):
        if words is not None:
            words[:] = torch.tensor([1, 3, 5, 9, 17] * 3)  # each its own and the first draft
            words[12] = 1  # sees nothing of the draft that is its own
        # sequence 0: drafts are tokens 43..47; draft 2 has NaN in three channels of head 0, draft 4 in all of head 1
        for c, code in ((0, 0x7F), (5, 0xFF), (dim - 1, 0x7F)):
            plant(codes, table, 0, 45, 1, 0, c, code)
        plant(codes, table, 0, 47, 1, 1, slice(None), 0x7F)
        # sequence 1: draft 1 (token 56) has a key that is NaN, draft 3 a value; a context token (3) a value in one channel
        plant(codes, table, 1, 56, 0, 0, 7, 0xFF)
        plant(codes, table, 1, 58, 1, 0, slice(10, 20), 0xFF)
        plant(codes, table, 1, 3, 1, 1, 33, 0x7F)
        # sequence 2: every place of draft 2 (token 63, the last of its page) and all past the end
        plant(codes, table, 2, 63, 0, slice(None), slice(None), 0x7F)
        plant(codes, table, 2, 63, 1, slice(None), slice(None), 0x7F)
        codes.view(torch.uint8)[int(table[2, 4]), :, :, 2:] = 0xFF
        scales[int(table[2, 4]), :, :, 2:] = float("nan")

    say("nan codes", group, dim, tree)
    cache_case(np.random.default_rng(41), "e4m3", 2, group, dim, 16, [48, 60, 66], 5, tree, touch=touch)


def test_nan_codes_among_many_rows():
    """Blocks of 256 rows: 64 drafts of which some are NaN."""
    def touch(codes, scales, table, rq, words):
        for seq, token in ((0, 300 - 64 + 10), (0, 299), (1, 1100 - 30)):
            plant(codes, table, seq, token, 1, slice(None), slice(3, 90), 0x7F)
        plant(codes, table, 1, 1100 - 64, 0, 1, 0, 0xFF)

    cache_case(np.random.default_rng(42), "e4m3", 2, 128, 128, 16, [300, 1100], 64, True, touch=touch, some=6)


def test_padded_drafts_over_a_cache_that_was_never_cleared():
    """A tree of three padded to eight with slots of -1, in memory that holds 0x7f everywhere."""
    rng = np.random.default_rng(43)
    codes = torch.full((8, 2, 2, 16, 128), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.full((8, 2, 2, 16), 1.0, dtype=torch.float32, device="cuda")
    table = ints([[5, 2, 7]])
    k, v, rq = rows(rng, 33, 2, 128), rows(rng, 33, 2, 128), rows(rng, 8, 8, 128)
    slot = [int(table[0, t // 16]) * 16 + t % 16 for t in range(33)]
    q().qcache_write(k, v, torch.tensor(slot, device="cuda"), codes, scales)
    words = torch.tensor([1, 3, 5, 0, 0, 0, 0, 0], dtype=torch.int64, device="cuda")
    got = f64(q().qattn_cache(rq, codes, scales, table, ints([38]), cu_q=ints([0, 8]), tree=words))
    c, s = ref.quantise(np.stack([k.float().cpu().numpy(), v.float().cpu().numpy()]), "e4m3")
    val = ref.code_values(c, "e4m3") * s.astype(np.float64)[..., None]
    for i in range(8):
        sees = ref.cache_sees(i, 8, 38, int(words[i]))
        for h in range(8):
            o, bound = ref.attend(f64(rq)[i, h], val[0][:, h // 4], val[1][:, h // 4], sees, 128 ** -0.5)
            check(got[i, h], o, bound, "row %d head %d" % (i, h))


# ---------------------------------------------------------------- counters ---
def test_graphs_of_one_stream_replayed_on_others():
    """Two graphs captured on one stream, of two and of three calls that join parts, replayed in turn on other streams,
    with eager calls on the first between them: ordered by events, each gives the eager call's bits every time."""
    rng = np.random.default_rng(51)
    codes, scales = random_cache(rng, "int8", 900, 16, 2, 128)
    lens = [6000, 5000, 40]
    table, n = tables(rng, lens, 16, 900), ints(lens)
    few, many = rows(rng, 3, 16, 128), rows(rng, 48, 32, 128)
    cu, cuq, cuk = starts([16, 20, 12]), starts([10, 4]), starts([2500, 1500])
    pq, pk = rows(rng, 14, 4, 128), rows(rng, 4000, 1, 128)
    wide = torch.full((3, (1 << 25) // (16 * 48 * 32) + 1), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    calls = [lambda: q().qattn_cache(few, codes, scales, table, n), lambda: q().qattn_prompt(pq, pk, pk, cuq, cuk),
             lambda: q().qattn_cache(many, codes, scales, wide, n, cu_q=cu)]
    home, away = torch.cuda.Stream(), [torch.cuda.Stream(), torch.cuda.Stream()]
    home.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(home):
        want = [bits(c()) for c in calls]
    graphs, outs = [], []
    for chain in ([0, 1, 2], [2, 0]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=home):
            outs.append([(i, calls[i]()) for i in chain])
        graphs.append(g)
    for turn in range(6):
        for i, out in outs[turn % 2]:
            out.fill_(3.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(away[turn % 2]):
            graphs[turn % 2].replay()
        home.wait_stream(away[turn % 2])
        with torch.cuda.stream(home):
            eager = [c() for c in calls[:1 + turn % 3]]
        torch.cuda.synchronize()
        for i, out in outs[turn % 2] + list(enumerate(eager)):
            assert np.array_equal(bits(out), want[i]), (turn, i)


# ------------------------------------------------- values that are not numbers ---
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("shape", ["whole tiles", "paired waves", "slices"])
def test_a_value_that_is_not_a_number_at_any_place(shape, dim):
    """NaN or an infinity in one channel of one value, at places on both sides of tile and block ends: rows that see it
    are not finite in that channel and right in the others, rows that do not are right."""
    rng = np.random.default_rng(61)
    nq, nk, heads, group = {"whole tiles": (1200, 1200, 2, 32), "paired waves": (300, 333, 1, 2),
                            "slices": (40, 2100, 1, 2)}[shape]
    rq, rk, rv = rows(rng, nq, heads * group, dim), rows(rng, nk, heads, dim), rows(rng, nk, heads, dim)
    off = nk - nq
    clean = f64(q().qattn_prompt(rq, rk, rv, starts([nq]), starts([nk])))
    kk, vv, qq = f64(rk), f64(rv), f64(rq)
    for at in (0, off + 1, off + 5, off + 31, off + 32, off + 33, nk - 64, nk - 2, nk - 1):
        bad = (float("nan"), float("inf"), -float("inf"))[at % 3]
        v = rv.clone()
        v[at, 0, 7] = bad
        got = f64(q().qattn_prompt(rq, rk, v, starts([nq]), starts([nk])))
        first = max(0, at - off)  # the first row that sees it
        for h in range(group):
            assert not np.isfinite(got[first:, h, 7]).any(), (at, h)
            assert np.isfinite(got[:first, h]).all() and np.isfinite(np.delete(got[first:, h], 7, axis=1)).all(), (at, h)
            assert np.array_equal(np.delete(got[first:, h], 7, axis=1), np.delete(clean[first:, h], 7, axis=1)), (at, h)
        assert np.array_equal(got[:, group:], clean[:, group:]), at
        for i in sorted({0, max(first - 1, 0), max(first - 17, 0), max(first - 40, 0)}):
            if i >= first:
                continue
            for h in (0, group - 1):
                o, bound = ref.attend(qq[i, h], kk[:, 0], vv[:, 0], np.arange(i + off + 1), dim ** -0.5)
                check(got[i, h], o, bound, "value %d row %d head %d" % (at, i, h))


@pytest.mark.parametrize("causal", [True, False])
def test_a_nan_that_rows_see_costs_no_second_pass(causal):
    """One NaN in the first value, or in the middle: the call takes about the time it takes without."""
    rng = np.random.default_rng(62)
    rq, rk, rv = rows(rng, 2048, 32, 128), rows(rng, 2048, 4, 128), rows(rng, 2048, 4, 128)
    cu = starts([2048])

    def time_of(v):
        best = []
        for _ in range(8):
            a, b = torch.cuda.Event(True), torch.cuda.Event(True)
            a.record()
            q().qattn_prompt(rq, rk, v, cu, causal=causal)
            b.record()
            b.synchronize()
            best.append(a.elapsed_time(b))
        return sorted(best)[3]

    clean = time_of(rv)
    for at in (0, 1024):
        v = rv.clone()
        v[at, :, 3] = float("nan")
        assert time_of(v) < 4 * clean


# ------------------------------------------------------------------- slots ---
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_a_slot_named_twice_touches_no_other(kind):
    """Tokens 0..99 again as 100..199 at the same slots (equal rows, so that the content is known), padding between:
    what these slots hold is right, and all others are as they were."""
    rng = np.random.default_rng(71)
    codes, scales = q().new_cache(14, 16, 3, 128, {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}[kind])
    codes.view(torch.uint8).fill_(0x5A)
    scales.fill_(-7.0)
    x = rows(rng, 100, 3, 128, torch.float32)
    twice = torch.cat([x, x])
    at = rng.permutation(14 * 16)[:100]
    slots = np.concatenate([at, at])
    slots[[7, 107, 50, 150]] = -1
    q().qcache_write(twice, -twice, torch.tensor(slots, device="cuda"), codes, scales)
    got_c, got_s = codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy()
    want_c, want_s = np.full_like(got_c, 0x5A), np.full_like(got_s, -7.0)
    for which, sign in ((0, 1), (1, -1)):
        c, s = ref.quantise(sign * x.cpu().numpy(), kind)
        for t, slot in enumerate(slots[:100]):
            if slot >= 0:
                want_c[slot // 16, which, :, slot % 16], want_s[slot // 16, which, :, slot % 16] = c[t], s[t]
    assert np.array_equal(got_s, want_s)
    assert np.array_equal(np.where(got_c == 0x80, 0, got_c), np.where(want_c == 0x80, 0, want_c))


# ----------------------------------------------------------------- strides ---
def test_dimensions_of_one_may_have_any_stride():
    """One token, or one head, with the strides that a transposed or expanded vector leaves there."""
    rng = np.random.default_rng(91)

    def odd(t, dim):  # the same values, a stride of 1 in a dimension of one
        strides = list(t.stride())
        strides[dim] = 1
        return t.as_strided(t.shape, strides)

    codes, scales = random_cache(rng, "int8", 4, 16, 1, 64)
    table = tables(rng, [40], 16, 4)
    one, k, v = rows(rng, 1, 4, 64), rows(rng, 9, 1, 64), rows(rng, 9, 1, 64)
    want = bits(q().qattn_cache(one, codes, scales, table, ints([40])))
    assert np.array_equal(want, bits(q().qattn_cache(odd(one, 0), codes, scales, table, ints([40]))))
    cu, cuk = starts([1]), starts([9])
    want = bits(q().qattn_prompt(one, k, v, cu, cuk))
    assert np.array_equal(want, bits(q().qattn_prompt(odd(one, 0), odd(k, 1), odd(v, 1), cu, cuk)))
    slots = torch.arange(9, device="cuda")
    for x in (k, k.float()):
        caches = [q().new_cache(1, 16, 1, 64) for _ in range(2)]
        q().qcache_write(x, x, slots, *caches[0])
        q().qcache_write(odd(x, 1), odd(x, 1), slots, *caches[1])
        assert torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])
    with pytest.raises(q().Qw3Error):
        wide = torch.zeros(2, 4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[:, :256].view(2, 4, 64)
        q().qattn_prompt(wide, k, v, starts([2]), cuk)
