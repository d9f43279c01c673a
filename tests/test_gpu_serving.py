"""The cache's calls together, as a server uses them: a decode step captured once
and replayed, with beams that part, against the same steps done one by one."""
import ctypes
import math
import sys

import numpy as np
import pytest
import torch

from oracle import attention as ref
from oracle import rope as rope_ref

pytestmark = pytest.mark.gpu


def q():
    import dequant_gemv_qgemv_amd as mod
    return mod


def say(*args):
    print("[gpu-case]", *args, file=sys.stderr, flush=True)


class Server:
    """One layer's cache of several sequences, all of whose state lives on the GPU."""

    def __init__(self, beams, heads, kv, dim, pages, size, width, count):
        d = "cuda"
        self.size, self.count = size, count
        self.codes, self.scales = q().new_cache(pages, size, kv, dim)
        self.bounds = q().new_bounds(self.codes)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=d)
        self.table = torch.full((beams, width), -1, dtype=torch.int32, device=d)
        self.lens = torch.zeros(beams, dtype=torch.int32, device=d)
        self.parents = torch.arange(beams, dtype=torch.int32, device=d)
        self.rates = torch.tensor(1000.0 ** (-np.arange(dim // 2) / (dim // 2)), device=d)
        self.q = torch.zeros(beams, heads, dim, device=d)
        self.k, self.v = torch.zeros(beams, kv, dim, device=d), torch.zeros(beams, kv, dim, device=d)

    def step(self):
        """Every beam follows its parent and takes one more token."""
        m = q()
        table, lens = m.qcache_fork(self.refs, self.table, self.lens, self.parents, self.size)
        positions = lens.clone()
        slots, lens, copies = m.qcache_reserve(self.refs, table, lens, self.size)
        m.qcache_copy(self.codes, self.scales, copies)
        x = m.qrope_write(self.q, self.k, self.v, positions, self.rates, slots, self.codes, self.scales)
        m.qcache_bounds(self.codes, self.scales, table, lens, *self.bounds)
        picks = m.qblock_select(x, *self.bounds, table, lens, self.count, self.size)
        out = m.qattn_blocks(x, self.codes, self.scales, table, lens, picks)
        self.table.copy_(table)
        self.lens.copy_(lens)
        return out, picks, slots

    def state(self):
        return [t.clone() for t in (self.codes, self.scales, *self.bounds, self.refs, self.table, self.lens)]


def test_captured_decode_with_beams():
    rng = np.random.default_rng(31)
    beams, heads, kv, dim, size, width, count, steps = 6, 8, 2, 64, 16, 8, 4, 90
    one, two = (Server(beams, heads, kv, dim, 60, size, width, count) for _ in range(2))
    # captured on one server, whose state is put back afterwards
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        one.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = one.step()
    for t, fresh in zip((one.codes, one.scales, *one.bounds, one.refs, one.table, one.lens), two.state()):
        t.copy_(fresh)
    history = [[] for _ in range(beams)]  # the tokens of each beam, as (step, beam)
    tokens = {}
    for step in range(steps):
        say("step", step)
        parents = rng.integers(0, beams, beams) if step % 7 == 3 else np.arange(beams)
        x = [torch.tensor(rng.standard_normal((beams, n, dim)), dtype=torch.float32) for n in (heads, kv, kv)]
        for s in (one, two):
            for to, new in zip((s.q, s.k, s.v), x):
                to.copy_(new)
            s.parents.copy_(torch.tensor(parents))
        graph.replay()
        eager = two.step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
        assert all(torch.equal(a, b) for a, b in zip(one.state(), two.state()))
        history = [history[p] + [(step, b)] for b, p in enumerate(parents)]
        for b in range(beams):
            tokens[step, b] = x[0][b].numpy(), x[1][b].numpy(), x[2][b].numpy()
        # nobody's page is anybody else's
        names = two.table[two.table >= 0].cpu().numpy()
        assert np.array_equal(two.refs.cpu().numpy(), np.bincount(names, minlength=60))
        assert two.lens.tolist() == [step + 1] * beams
        if step % 15 != 14:
            continue
        # a beam's output against attention over its own tokens, of the pages picked
        got, picks = eager[0].float().cpu().numpy(), eager[1].cpu().numpy()
        rates = two.rates.cpu().numpy()
        for b in (0, beams - 1):
            at = np.arange(step + 1)
            keys = np.stack([tokens[t][1] for t in history[b]])
            keys = rope_ref.rotate(keys, at[None], rates, np.zeros(len(rates), int), "halves")[0]
            values = np.stack([tokens[t][2] for t in history[b]]).astype(np.float64)
            query = rope_ref.rotate(tokens[history[b][-1]][0][None], np.array([[step]]), rates, np.zeros(len(rates), int), "halves")[0][0]
            for h in range(kv):
                mine = picks[b, h][picks[b, h] >= 0]
                assert len(mine) == min(count, step // size + 1) and mine[-1] == step // size
                seen = np.concatenate([np.arange(p * size, min((p + 1) * size, step + 1)) for p in mine])
                for g in range(h * heads // kv, (h + 1) * heads // kv):
                    want, _ = ref.attend(query[g], keys[:, h], values[:, h], seen, 1 / math.sqrt(dim))
                    # a score is off by the int8 keys' half steps (max|k| / 254) and the bf16 query's 2^-8, a weight by
                    # exp of twice that, a value by its own half step, the output by 2^-8
                    score = (np.abs(query[g]).sum() * np.abs(keys).max() / 254 + 2.0 ** -8 * (np.abs(keys[seen, h]) @ np.abs(query[g])).max()) / math.sqrt(dim)
                    top = np.abs(values).max()
                    bound = top * (np.exp(2 * score) - 1) + top / 254 + 2.0 ** -8 * np.abs(want) + 1e-4
                    assert np.all(np.abs(got[b, g] - want) <= bound)


def test_sequences_that_get_no_room_write_nothing():
    """A pool that is too small: slots of -1 all the way through, the other sequences as if they were alone."""
    size, kv, dim = 16, 2, 64
    codes, scales = q().new_cache(3, size, kv, dim)
    refs = torch.zeros(3, dtype=torch.int32, device="cuda")
    table = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 20, 40, 45], dtype=torch.int32, device="cuda")  # 2 + 2 + 1 pages
    slots, after, copies = q().qcache_reserve(refs, table, lens, size, cu=cu, total=45)
    assert after.tolist() == [20, 0, 0] and (slots[:20] >= 0).all() and (slots[20:] == -1).all() and (copies == -1).all()
    assert refs.sum() == 2
    x = torch.randn(45, kv, dim, device="cuda")
    rates = torch.full((dim // 2,), 0.1, dtype=torch.float64, device="cuda")
    positions = torch.arange(45, dtype=torch.int32, device="cuda")
    q().qrope_write(x, x, x, positions, rates, slots, codes, scales)
    assert int((scales != 0).sum()) == 20 * 2 * kv
    out = q().qattn_cache(x.to(torch.bfloat16), codes, scales, table, after, cu_q=cu)
    assert (out[20:] == 0).all() and (out[:20] != 0).any(dim=2).all()


def test_a_capture_that_would_allocate_is_refused():
    """On a stream that has not run the calls at their size a capture is refused, and nothing is enqueued; after one call it is taken."""
    m = q()
    with open("/proc/self/maps") as maps:  # the runtime that is loaded, and no other copy
        hip = ctypes.CDLL(next(line.split()[-1] for line in maps if "libamdhip64" in line))
    size, heads, dim, width = 16, 2, 64, 1500
    codes, scales = m.new_cache(2 * width, size, heads, dim)
    bounds = m.new_bounds(codes)
    table = torch.arange(2 * width, dtype=torch.int32, device="cuda").view(2, width)
    lens = torch.full((2,), width * size, dtype=torch.int32, device="cuda")
    x = torch.randn(2, 4, dim, device="cuda").to(torch.bfloat16)
    picks = torch.arange(40, dtype=torch.int32, device="cuda").expand(2, heads, 40).contiguous()
    keep = torch.ones(2 * width * size, dtype=torch.bool, device="cuda")
    cu = torch.tensor([0, width * size, 2 * width * size], dtype=torch.int32, device="cuda")
    calls = [lambda: m.qblock_select(x, *bounds, table, lens, 40, size), lambda: m.qattn_blocks(x, codes, scales, table, lens, picks),
             lambda: m.qcache_compact(codes, scales, table, lens, keep, cu_q=cu)]
    for call in calls:
        call()  # the kernels are loaded; on another stream than below
        torch.cuda.synchronize()
        handle = ctypes.c_void_p()  # torch's own streams are used again and again; this one is nobody else's
        assert hip.hipStreamCreate(ctypes.byref(handle)) == 0
        side, graph = torch.cuda.ExternalStream(handle.value), torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                still = lens + 0
                with pytest.raises(m.Qw3Error) as refused:
                    call()
            assert refused.value.status == m.QW3_ERR_CAPTURE
            graph.replay()
            assert torch.equal(still, lens)
            want = call()
            side.synchronize()
            again = torch.cuda.CUDAGraph()
            with torch.cuda.graph(again, stream=side):
                got = call()
            again.replay()
            side.synchronize()
            assert torch.equal(got, want)
