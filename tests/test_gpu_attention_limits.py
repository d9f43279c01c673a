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
