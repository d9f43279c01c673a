"""Host threads that call on one stream at once: calls of several launches pass data
through the stream's buffer, and each has to find its own.  The expected results are
those of the same calls one after the other."""
import threading

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def q():
    import dequant_gemv_qgemv_amd as mod
    return mod


def compaction(seed, tokens):
    """A call that drops some of a context's tokens, many launches' worth, and what it leaves."""
    rng = np.random.default_rng(seed)
    size, heads, dim, layers = 16, 4, 64, 2
    pages = -(-tokens // size)
    raw = torch.tensor(rng.integers(0, 256, (layers, pages, 2, heads, size, dim), dtype=np.uint8)).cuda()
    scale = torch.tensor(rng.random((layers, pages, 2, heads, size), dtype=np.float32)).cuda()
    table = torch.tensor(rng.permutation(pages)[None].astype(np.int32)).cuda()
    keep = torch.tensor(rng.random(tokens) < 0.6).cuda()
    lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([tokens], [0, tokens]))

    def call():
        codes, scales = raw.clone().view(torch.int8), scale.clone()
        return q().qcache_compact(codes, scales, table, lens, keep, cu_q=cu), codes, scales
    return call


def selection(seed, n):
    rng = np.random.default_rng(seed)
    size, heads, dim = 16, 2, 128
    pages = -(-n // size)
    limits = torch.tensor(rng.integers(-127, 128, (pages, heads, 2, dim)).astype(np.int8)).cuda()
    steps = torch.tensor(rng.random((pages, heads), dtype=np.float32)).cuda()
    x = torch.tensor(rng.standard_normal((3, 8, dim)), dtype=torch.float32).to(torch.bfloat16).cuda()
    table = torch.tensor(rng.permutation(pages)[None].astype(np.int32)).cuda()
    lens, cu = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([n], [0, 3]))
    return lambda: (q().qblock_select(x, limits, steps, table, lens, 24, size, cu_q=cu),)


def product(seed, rows):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    codes = torch.randint(0, 8, (512, 8192), dtype=torch.uint8, device="cuda", generator=g)
    packed = q().qpack_uint3(codes)
    scales = torch.rand(512, 64, device="cuda", generator=g).to(torch.bfloat16)
    x = torch.randn(rows, 8192, device="cuda", generator=g).to(torch.bfloat16)
    return lambda: (q().qgemm_w3g128_smallM(x, packed, scales),)


def test_threads_on_one_stream():
    calls = [compaction(1, 3000), compaction(2, 5000), selection(3, 50000), product(4, 40), product(5, 300)]
    want = [call() for call in calls]  # the buffer has its size from here on
    torch.cuda.synchronize()
    got, errors = [[] for _ in calls], []
    ready = threading.Barrier(len(calls))

    def work(i):
        try:
            ready.wait(30)
            for _ in range(15):
                got[i].append(calls[i]())
        except Exception as e:  # reported below, by the test's own thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for mine, all_of in zip(want, got):
        assert len(all_of) == 15
        for each in all_of:
            assert all(torch.equal(a, b) for a, b in zip(mine, each))
