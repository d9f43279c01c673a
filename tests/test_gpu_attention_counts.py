"""Every key counts once: attention on the GPU with queries of zero, where an output
is the share of the row's keys with a one in its channel (oracle/attention.py), over
the lengths at which work is split; and weights of two bf16 where they are promised."""
import functools

import numpy as np
import pytest
import torch

from oracle import attention as ref
from test_gpu_attention import TORCH, cache_case, check, f64, q, random_cache, rows, say, starts, tables

pytestmark = pytest.mark.gpu
ONE = {"int8": 1, "e4m3": 0x38}


def cache_counts(rng, kind, heads, group, dim, page, lens, news, tree, wide=0):
    """`wide`: keys that the table can name, for the kernels of large calls."""
    pages = sum(-(-n // page) for n in lens) + 2
    codes, scales = random_cache(rng, kind, pages, page, heads, dim)
    scales[:, 1] = 1.0
    raw = codes.view(torch.uint8)
    raw[:, 1] = 0x7E  # what is not a token of the sequences is large
    table = tables(rng, lens, page, pages)
    if wide:
        t = torch.full((len(lens), wide // page), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
        t[:, :table.shape[1]] = table
        table = t
    rq = torch.zeros(sum(news), heads * group, dim, dtype=torch.bfloat16, device="cuda")
    words = torch.tensor(rng.integers(-2 ** 63, 2 ** 63, sum(news)), dtype=torch.int64) if tree else None
    tab = table.cpu().numpy()
    parts = ref.counting_parts(max(lens), dim)
    for part in range(parts):
        values = []
        for b, n in enumerate(lens):
            values.append([ref.counting_values(n, dim, (part + h) % parts, parts) for h in range(heads)])
            at = torch.arange(n, device="cuda")
            page_of = torch.tensor(tab[b], device="cuda").long()[at // page]
            for h in range(heads):
                raw[page_of, 1, h, at % page] = torch.tensor(values[b][h] * ONE[kind], dtype=torch.uint8, device="cuda")
        got = f64(q().qattn_cache(rq, codes, scales, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                  cu_q=starts(news), tree=words.cuda() if tree else None))
        at = 0
        for b, (n, length) in enumerate(zip(news, lens)):
            seen = np.zeros((n, length), bool)
            for i in range(n):
                seen[i, ref.cache_sees(i, n, length, int(words[at + i]) & (2 ** 64 - 1) if tree else None)] = True
            for h in range(heads * group):
                bad = ref.miscounted(got[at:at + n, h], seen, values[b][h // group])
                assert not bad.any(), "part %d sequence %d head %d: rows and channels %s" % (part, b, h, np.argwhere(bad)[:5])
            at += n


@pytest.mark.parametrize("kind,heads,group,dim,page,lens,news,tree", [
    ("int8", 1, 8, 128, 16, [20000], [1], False),                 # one head cut for the card
    ("int8", 2, 4, 128, 64, [30000, 5, 9001], [1, 1, 1], False),
    ("e4m3", 1, 4, 64, 16, [12345, 700], [4, 2], True),
    ("e4m3", 8, 8, 128, 16, [129, 1, 0, 2048, 127, 4000], [1] * 6, False),
    ("int8", 2, 8, 128, 16, [9000, 33], [4, 3], True),            # blocks of 32
    ("e4m3", 1, 8, 64, 32, [7001, 257, 64], [5, 8, 2], False),
    ("int8", 2, 2, 64, 128, [131, 5000], [13, 13], True),
    ("int8", 1, 8, 128, 16, [1500], [64], True),                  # small call, many rows
], ids=str)
def test_few_rows(kind, heads, group, dim, page, lens, news, tree):
    say("counts", kind, heads, group, dim, lens, news, tree)
    cache_counts(np.random.default_rng(81), kind, heads, group, dim, page, lens, news, tree)


@pytest.mark.parametrize("kind,heads,group,dim,page,lens,news,tree", [
    ("int8", 1, 8, 64, 16, [6000, 100], [64, 40], True),            # blocks of 128
    ("e4m3", 2, 4, 64, 32, [129, 3000, 64], [30, 40, 30], False),
    ("int8", 1, 16, 128, 16, [5000], [8], True),
    ("e4m3", 2, 128, 128, 64, [900, 4100], [64, 64], True),         # blocks of 256
], ids=str)
def test_many_rows(kind, heads, group, dim, page, lens, news, tree):
    say("counts", kind, heads, group, dim, lens, news, tree)
    wide = (1 << 25) // (sum(news) * heads * group) // page * page + page
    cache_counts(np.random.default_rng(82), kind, heads, group, dim, page, lens, news, tree, max(wide, 8192))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nq,nk,heads,group", [
    ([1200, 1], [1200, 1], 2, 32),              # tiles of 128 rows
    ([300, 31, 64], [300, 31, 64], 1, 3),       # paired waves
    ([20, 130], [6000, 131], 1, 4),             # slices
    ([1], [30000], 1, 1), ([100, 3], [2049, 4000], 2, 1),
    ([70, 5, 0] * 30, [90, 5, 3] * 30, 1, 2),   # more sequences than lanes
], ids=["whole tiles", "paired waves", "slices", "one row", "uneven slices", "many"])
def test_prompts(causal, dim, nq, nk, heads, group):
    say("counts", causal, dim, nq[:6], nk[:6])
    rng = np.random.default_rng(83)
    rk = rows(rng, sum(nk), heads, dim)
    rq = torch.zeros(sum(nq), heads * group, dim, dtype=torch.bfloat16, device="cuda")
    parts = ref.counting_parts(max(nk), dim)
    for part in range(parts):
        values = [ref.counting_values(n, dim, part, parts) for n in nk]
        rv = torch.tensor(np.concatenate(values), device="cuda").bfloat16()[:, None].expand(-1, heads, -1).contiguous()
        got = f64(q().qattn_prompt(rq, rk, rv, starts(nq), starts(nk), causal=causal))
        at = 0
        for b, (n, length) in enumerate(zip(nq, nk)):
            i, j = np.arange(n)[:, None], np.arange(length)[None]
            seen = (j <= i + length - n) if causal else np.ones((n, length), bool)
            for h in range(heads * group) if b < 6 else ():
                bad = ref.miscounted(got[at:at + n, h], seen, values[b])
                assert not bad.any(), "part %d sequence %d head %d: rows and channels %s" % (part, b, h, np.argwhere(bad)[:5])
            at += n


# ------------------------------------------------------ weights of two bf16 ---
@pytest.mark.parametrize("kind,heads,group,dim,page,lens,news,tree", [
    ("int8", 2, 8, 128, 16, [300, 47, 1000], [1, 1, 1], False), ("e4m3", 2, 4, 64, 32, [129, 500], [3, 4], True),
    ("int8", 1, 8, 128, 16, [90, 64], [4, 8], True), ("e4m3", 1, 8, 128, 16, [200, 333], [6, 7], False),
    ("int8", 1, 4, 64, 16, [5000], [2], True)], ids=str)
def test_few_rows_keep_two_bf16(kind, heads, group, dim, page, lens, news, tree, monkeypatch):
    """The bound with 2^-16 for a weight in place of 2^-8."""
    monkeypatch.setattr(ref, "attend", functools.partial(ref.attend, weight_error=2.0 ** -16))
    cache_case(np.random.default_rng(84), kind, heads, group, dim, page, lens, news, tree)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group,new", [(1, 1), (8, 4), (8, 40)])
def test_a_weight_half_way_between_two_bf16(group, new, dim):
    """Two kinds of keys whose values cancel: one bf16 for a weight is 20 times the bound off. `new` of 40: the small
    call of many rows."""
    n = 200
    codes, scales = q().new_cache(13, 16, 1, dim, TORCH["int8"])
    table = torch.arange(13, dtype=torch.int32, device="cuda").view(1, -1)
    k, v = torch.zeros(n, 1, dim, device="cuda"), torch.ones(n, 1, dim, device="cuda")
    k[100:, :, 0] = ref.HALF_WAY
    v[:100] = -np.exp(ref.HALF_WAY)
    q().qcache_write(k, v, torch.arange(n, device="cuda"), codes, scales)
    rq = torch.zeros(new, group, dim, dtype=torch.bfloat16, device="cuda")
    rq[:, :, 0] = 1.0
    words = torch.zeros(new, dtype=torch.int64, device="cuda")  # no draft is seen: 200 - new keys, half and half below
    got = f64(q().qattn_cache(rq, codes, scales, table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                              cu_q=starts([new]), tree=words, sm_scale=1.0))
    c, s = ref.quantise(np.stack([k.cpu().numpy(), v.cpu().numpy()]), "int8")
    val = c.view(np.int8).astype(np.float64) * s[..., None]
    for i in range(new):
        for h in range(group):
            o, bound = ref.attend(f64(rq)[i, h], val[0][:, 0], val[1][:, 0], np.arange(n - new), 1.0, 2.0 ** -16)
            check(got[i, h], o, bound, "row %d head %d" % (i, h))
