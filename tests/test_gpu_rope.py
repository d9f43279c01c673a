"""Rotary positions on the GPU against their definition in 64 bits
(oracle/rope.py), and what they write into the cache."""
import sys

import numpy as np
import pytest
import torch

from oracle import rope as ref

pytestmark = pytest.mark.gpu

TORCH = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def q():
    import dequant_gemv_qgemv_amd as mod
    return mod


def say(*args):
    print("[gpu-case]", *args, file=sys.stderr, flush=True)


def ints(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def angles(rng, tokens, pairs, axes, far):
    positions = rng.integers(-far, far + 1, (axes, tokens))
    positions[0, 0] = 0
    axis = rng.integers(0, axes, pairs)
    rates = 10000.0 ** (-np.arange(pairs) / pairs)
    return positions, rates, axis


def near(got, want, bound):
    """bf16 outputs: off by the bound, and by a rounding of 2^-8."""
    got = got.float().cpu().numpy().astype(np.float64)
    off = np.abs(got - want) - bound - 2.0 ** -8 * (np.abs(want) + bound) - 1e-37
    assert np.all(off <= 0), (float(off.max()), np.argwhere(off > 0)[:4])


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.uint8).cpu().numpy()


SHAPES = [  # tokens, heads, kv heads, channels, rotated, axes, farthest position
    (1, 1, 1, 64, 64, 1, 5), (1, 64, 8, 128, 128, 1, 131071), (3, 5, 5, 128, 128, 3, 900), (7, 8, 2, 64, 32, 2, 77),
    (70, 14, 2, 128, 48, 4, 2 ** 31 - 1), (33, 7, 1, 64, 16, 1, 1 << 20), (257, 64, 8, 128, 128, 3, 40000), (1027, 12, 4, 64, 48, 8, 3000)]


@pytest.mark.parametrize("style", ["halves", "pairs"])
@pytest.mark.parametrize("src", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rotation_and_cache(style, src, shape):
    say("rope", style, src, shape)
    tokens, heads, kv, dim, rotated, axes, far = shape
    rng = np.random.default_rng(tokens + heads)
    positions, rates, axis = angles(rng, tokens, rotated // 2, axes, far)
    gp, gr, ga = ints(positions), ints(rates, torch.float64), ints(axis)
    fused = torch.tensor(rng.standard_normal((tokens, heads + 2 * kv + 1, dim)), dtype=torch.float32).to(src).cuda()
    x, k, v = fused[:, :heads], fused[:, heads:heads + kv], fused[:, heads + kv + 1:]
    sample = np.unique(np.r_[0, tokens - 1, rng.integers(0, tokens, 12)])

    def want(t):
        return ref.rotate(t.float().cpu().numpy()[sample], positions[:, sample], rates, axis, style)

    got = q().qrope(x, gp, gr, axis=ga, style=style)
    assert got.shape == x.shape and got.dtype is torch.bfloat16 and got.is_contiguous()
    near(got[sample], *want(x))

    page = 16
    pages = -(-tokens // page) + 2
    for name, kind in TORCH.items():
        codes, scales = q().new_cache(pages, page, kv, dim, kind)
        codes.view(torch.uint8).fill_(0x5A)
        scales.fill_(-7.0)
        slots = rng.permutation(pages * page)[:tokens]
        if tokens > 6:
            slots[2], slots[4], slots[5] = -1, pages * page, 1 << 40
        slots = ints(slots, torch.int64)
        qo, ko, vo = q().qrope_write(x, k, v, gp, gr, slots, codes, scales, axis=ga, style=style, dense=True)
        only = q().qrope_write(x, k, v, gp, gr, slots, codes, scales, axis=ga, style=style)
        assert np.array_equal(bits(qo), bits(got)) and np.array_equal(bits(only), bits(got))
        near(ko[sample], *want(k))
        assert np.array_equal(bits(ko), bits(q().qrope(k, gp, gr, axis=ga, style=style)))
        assert np.array_equal(bits(vo), bits(v.to(torch.bfloat16)))
        # v as qcache_write stores it; places of no slot as they were
        other = codes.clone(), scales.clone()
        plain_codes, plain_scales = q().new_cache(pages, page, kv, dim, kind)
        plain_codes.view(torch.uint8).fill_(0x5A)
        plain_scales.fill_(-7.0)
        q().qcache_write(k, v, slots, plain_codes, plain_scales)
        assert np.array_equal(bits(other[0])[:, 1], bits(plain_codes)[:, 1])
        assert torch.equal(other[1][:, 1], plain_scales[:, 1])
        unused = (plain_scales == -7.0)
        assert torch.equal(other[1] == -7.0, unused)
        assert (other[0].view(torch.uint8)[unused] == 0x5A).all()
        # k: codes times scale stand for the rotated row, one step of the code off at most by half
        y, bound = want(k)
        flat_codes = codes.view(torch.uint8)[:, 0].transpose(1, 2).reshape(-1, kv, dim).view(kind).float().cpu().numpy().astype(np.float64)
        flat_scales = scales[:, 0].transpose(1, 2).reshape(-1, kv).cpu().numpy().astype(np.float64)
        limit = 127 if name == "int8" else 448
        for i, t in enumerate(sample):
            at = int(slots[t])
            if not 0 <= at < pages * page:
                continue
            s = flat_scales[at][:, None]
            top = np.abs(y[i]).max(-1, keepdims=True)
            slack = bound[i].max(-1, keepdims=True)
            assert np.all(np.abs(s * limit - top) <= slack + 2.0 ** -23 * top)
            # half a step of the code, what the row is off, and c s with s off by what top is
            half = s / 2 if name == "int8" else np.maximum(2.0 ** -4 * np.abs(y[i]), s * 2.0 ** -10)
            off = np.abs(flat_codes[at] * s - y[i])
            assert np.all(off <= half * (1 + 2.0 ** -20) + 2 * slack + 2.0 ** -22 * top)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("src", [torch.float32, torch.bfloat16])
def test_position_zero_writes_what_qcache_write_does(kind, src):
    """Angle 0 turns nothing: keys, special ones among them, are stored bit for bit as qcache_write stores them."""
    rng = np.random.default_rng(4)
    tokens, kv, dim = 40, 3, 128
    k = torch.tensor(rng.standard_normal((tokens, kv, dim)), dtype=torch.float32)
    k[0, 0] = 0.0
    k[1, 0] *= 1e-30
    k[2, 1] *= 1e30
    k[3, 0, 5:] = 0.0
    k = k.to(src).cuda()
    v = torch.randn(tokens, kv, dim, device="cuda").to(src)
    v[4, 0, 3], v[5, 1, 9] = float("inf"), float("nan")
    slots = torch.arange(tokens, device="cuda")
    a, b = q().new_cache(4, 16, kv, dim, TORCH[kind]), q().new_cache(4, 16, kv, dim, TORCH[kind])
    rates = torch.full((64,), 0.3, dtype=torch.float64, device="cuda")
    zero = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    for style in ("halves", "pairs"):
        q().qrope_write(k, k, v, zero, rates, slots, *a, style=style)
        q().qcache_write(k, v, slots, *b)
        assert np.array_equal(bits(a[0]) & 0x7F if kind == "e4m3" else bits(a[0]), bits(b[0]) & 0x7F if kind == "e4m3" else bits(b[0]))
        assert torch.equal(torch.nan_to_num(a[1], -3.0), torch.nan_to_num(b[1], -3.0))


def test_rows_that_hold_no_numbers_stay_visible():
    x = torch.ones(3, 2, 64, device="cuda")
    x[0, 0, 3], x[1, 1, 40] = float("nan"), float("inf")
    pos = torch.arange(3, dtype=torch.int32, device="cuda") + 1
    rates = torch.full((16,), 0.7, dtype=torch.float64, device="cuda")
    codes, scales = q().new_cache(1, 16, 2, 64)
    got = q().qrope_write(x, x, x, pos, rates, torch.arange(3, device="cuda"), codes, scales).float()
    bad = torch.zeros(3, 2, 64, dtype=torch.bool, device="cuda")
    bad[0, 0, 3] = bad[0, 0, 19] = bad[1, 1, 40] = True
    assert torch.equal(~torch.isfinite(got), bad)
    scales = scales[0].transpose(1, 2)[:, :3]
    assert torch.equal(torch.isnan(scales), torch.stack([bad.any(-1)] * 2))


def test_two_dimensions_of_positions_and_no_axis():
    """[T] and [1, T] are the same; without `axis` every pair is on axis 0; an axis outside counts as the nearest."""
    x = torch.randn(9, 4, 128, device="cuda")
    rates = torch.tensor(10000.0 ** (-np.arange(64) / 64), device="cuda")
    p = torch.randint(0, 5000, (2, 9), dtype=torch.int32, device="cuda")
    one = q().qrope(x, p[0], rates)
    assert torch.equal(one, q().qrope(x, p[:1], rates))
    assert torch.equal(one, q().qrope(x, p, rates))
    assert torch.equal(one, q().qrope(x, p, rates, axis=torch.full((64,), -5, dtype=torch.int32, device="cuda")))
    last = q().qrope(x, p[1], rates)
    assert torch.equal(last, q().qrope(x, p, rates, axis=torch.full((64,), 1 << 30, dtype=torch.int32, device="cuda")))


def test_strides_outputs_and_rows_behind():
    """Views with other strides, one dimension of one, `out`, and rows behind the last token left as they were."""
    base = torch.randn(6, 130, 9, 64, device="cuda")
    rates = torch.full((32,), 0.01, dtype=torch.float64, device="cuda")
    p = torch.arange(130, dtype=torch.int32, device="cuda")
    x = base[3].transpose(0, 1).contiguous().transpose(0, 1)  # heads before tokens in memory
    want = q().qrope(base[3].contiguous(), p, rates)
    assert torch.equal(q().qrope(x, p, rates), want)
    assert torch.equal(q().qrope(base[3, :, :4], p, rates), want[:, :4])
    guard = torch.full((132, 9, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    assert q().qrope(x, p, rates, out=guard[:130]).data_ptr() == guard.data_ptr()
    assert torch.equal(guard[:130], want) and (guard[130:] == 5).all()
    one = base[0, :1, :1].transpose(0, 1)  # strides of dimensions of one may be anything
    assert torch.equal(q().qrope(one, p[3:4], rates)[0, 0], q().qrope(base[0, :1], p[3:4], rates)[0, 0])
    assert q().qrope(x[:0], p[:0], rates).shape == (0, 9, 64)


def test_replay_and_another_stream():
    """Captured once, replayed with other positions and inputs; the same on a stream of its own."""
    x = torch.randn(20, 6, 128, device="cuda")
    k = torch.randn(20, 2, 128, device="cuda")
    p = torch.zeros(2, 20, dtype=torch.int32, device="cuda")
    axis = (torch.arange(64, device="cuda") % 2).to(torch.int32)
    rates = torch.tensor(10000.0 ** (-np.arange(64) / 64), device="cuda")
    slots = torch.arange(20, device="cuda")
    codes, scales = q().new_cache(2, 16, 2, 128)

    def call():
        return q().qrope_write(x, k, k, p, rates, slots, codes, scales, axis=axis, dense=True)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(4):
        x.normal_(), k.normal_()
        p.copy_(torch.randint(0, 9999, (2, 20), device="cuda"))
        slots.copy_(torch.randperm(32, device="cuda")[:20])
        codes.zero_(), scales.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out] + [codes.clone(), scales.clone()]
        codes.zero_(), scales.zero_()
        want = list(call()) + [codes, scales]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        codes.zero_(), scales.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again = list(call()) + [codes, scales]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_refusals():
    x = torch.zeros(3, 4, 64, device="cuda")
    p, r = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(32, dtype=torch.float64, device="cuda")
    codes, scales = q().new_cache(2, 16, 2, 64)
    s = torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in (lambda: q().qrope(x, p, r, style="half"), lambda: q().qrope(x, p[:2], r), lambda: q().qrope(x, p, r[None]),
                lambda: q().qrope(x, p, r, axis=p), lambda: q().qrope(x.transpose(1, 2), p, r),
                lambda: q().qrope(x, p, r, out=torch.empty(3, 4, 64, device="cuda")),
                lambda: q().qrope_write(x, x[:, :2], x[:, :1], p, r, s, codes, scales),
                lambda: q().qrope_write(x[:, :3], x[:, :2], x[:, :2], p, r, s, codes, scales),
                lambda: q().qrope_write(x, x[:, :2], x[:, :2], p, r, s[:2], codes, scales),
                lambda: q().qrope_write(x, x[:2, :2], x[:2, :2], p, r, s, codes, scales)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q().qrope(x, p.long(), r), lambda: q().qrope(x, p, r.float()), lambda: q().qrope(x.half(), p, r),
                lambda: q().qrope_write(x, x[:, :2].bfloat16(), x[:, :2], p, r, s, codes, scales)):
        with pytest.raises(TypeError):
            bad()
    for rates in (r[:4], torch.zeros(40, dtype=torch.float64, device="cuda"), r[:0]):
        with pytest.raises(q().Qw3Error) as e:
            q().qrope(x, p, rates)
        assert e.value.status == q().QW3_ERR_SHAPE
