"""CPU checks of the cache and attention calls: bad arguments are refused on the
host, by the C entry points and by the binding.  Pointers here are fake and never
dereferenced: every call fails validation or has no work."""

import pytest
import torch

import dequant_gemv_qgemv_amd as q

A = [0x10000 * (i + 1) for i in range(10)]
NULL = None
S = None


def write(k=A[0], v=A[1], src=0, slots=A[2], codes=A[3], scales=A[4], kind=0, T=4, H=2, D=128, pages=8, size=16,
          kts=256, khs=128, vts=256, vhs=128):
    return q.raw().qcache_write(k, v, src, slots, codes, scales, kind, T, H, D, pages, size, kts, khs, vts, vhs, S)


def read(codes=A[0], scales=A[1], kind=0, table=A[2], cu=A[3], k=A[4], v=A[5], B=2, maxp=4, total=7, H=2, D=128,
         pages=8, size=16):
    return q.raw().qcache_read(codes, scales, kind, table, cu, k, v, B, maxp, total, H, D, pages, size, S)


def cache(qq=A[0], codes=A[1], scales=A[2], kind=0, table=A[3], lens=A[4], cu=A[5], tree=NULL, out=A[6], B=2, maxp=4,
          Tq=6, Hq=8, H=2, D=128, pages=8, size=16, ts=1024, hs=128, sm=0.1):
    return q.raw().qattn_cache(qq, codes, scales, kind, table, lens, cu, tree, out, B, maxp, Tq, Hq, H, D, pages, size,
                               ts, hs, sm, S)


def prompt(qq=A[0], k=A[1], v=A[2], cu_q=A[3], cu_k=A[4], out=A[5], B=2, Tq=6, Tk=9, Hq=8, H=2, D=128, qts=1024,
           qhs=128, kts=256, khs=128, vts=256, vhs=128, causal=1, sm=0.1):
    return q.raw().qattn_prompt(qq, k, v, cu_q, cu_k, out, B, Tq, Tk, Hq, H, D, qts, qhs, kts, khs, vts, vhs, causal,
                                sm, S)


CACHE_SHAPES = [dict(kind=2), dict(kind=-1), dict(H=0), dict(H=1 << 20), dict(D=96), dict(D=256), dict(size=8),
                dict(size=48), dict(size=131072), dict(pages=-1)]


@pytest.mark.parametrize("bad", CACHE_SHAPES, ids=str)
@pytest.mark.parametrize("call", [write, read, cache])
def test_cache_shapes(call, bad):
    assert call(**bad) == q.QW3_ERR_SHAPE


@pytest.mark.parametrize("call,bad", [
    (write, dict(src=2)), (write, dict(T=-1)), (write, dict(T=1 << 40)),
    (read, dict(B=-1)), (read, dict(B=1 << 20)), (read, dict(total=-1)), (read, dict(total=1 << 31)), (read, dict(maxp=-1)),
    (cache, dict(B=-1)), (cache, dict(B=1 << 20)), (cache, dict(Tq=-1)), (cache, dict(Tq=1 << 27)), (cache, dict(Hq=7)),
    (cache, dict(Hq=0)), (cache, dict(maxp=-1)), (cache, dict(maxp=1 << 27)), (cache, dict(sm=0.0)), (cache, dict(sm=-1.0)),
    (cache, dict(B=60000, Tq=1 << 20, maxp=1 << 20)),  # more work than is counted in 31 bits
    (cache, dict(sm=float("inf"))), (cache, dict(sm=float("nan"))), (cache, dict(ts=-8)), (cache, dict(cu=NULL)),
    (prompt, dict(D=80)), (prompt, dict(H=0)), (prompt, dict(Hq=9)), (prompt, dict(B=-1)), (prompt, dict(B=1 << 20)),
    (prompt, dict(Tq=-1)), (prompt, dict(Tk=-1)), (prompt, dict(Tk=1 << 27)), (prompt, dict(sm=0.0)),
    (prompt, dict(sm=float("nan"))), (prompt, dict(kts=-256)), (prompt, dict(kts=1 << 23)), (prompt, dict(vhs=-8))], ids=str)
def test_shapes(call, bad):
    assert call(**bad) == q.QW3_ERR_SHAPE


@pytest.mark.parametrize("call,bad", [
    (write, dict(T=1 << 62, H=4)), (write, dict(T=(1 << 63) - 1, H=1024)), (cache, dict(maxp=1 << 60)),
    (cache, dict(maxp=(1 << 63) - 1)), (cache, dict(maxp=1 << 58, size=64))], ids=str)
def test_sizes_whose_product_passes_64_bits(call, bad):
    assert call(**bad) == q.QW3_ERR_SHAPE


@pytest.mark.parametrize("call,names", [
    (write, ("k", "v", "slots", "codes", "scales")), (read, ("codes", "scales", "table", "cu", "k", "v")),
    (cache, ("qq", "codes", "scales", "table", "lens", "out")), (prompt, ("qq", "k", "v", "cu_q", "cu_k", "out"))])
def test_null_pointers(call, names):
    for name in names:
        assert call(**{name: NULL}) == q.QW3_ERR_NULL, name


@pytest.mark.parametrize("call,bad", [
    (write, dict(k=0x10008)), (write, dict(codes=0x10008)), (write, dict(scales=0x10004)), (write, dict(slots=0x10004)),
    (write, dict(kts=252)), (write, dict(vhs=4)), (write, dict(src=1, khs=2)),
    (read, dict(codes=0x10008)), (read, dict(table=0x10002)), (read, dict(cu=0x10001)), (read, dict(k=0x10008)),
    (cache, dict(qq=0x10008)), (cache, dict(out=0x10008)), (cache, dict(lens=0x10002)), (cache, dict(cu=0x10002)),
    (cache, dict(tree=0x10004)), (cache, dict(ts=1020)), (cache, dict(hs=4)),
    (prompt, dict(qq=0x10008)), (prompt, dict(v=0x10008)), (prompt, dict(out=0x10004)), (prompt, dict(cu_k=0x10002)),
    (prompt, dict(qhs=4)), (prompt, dict(kts=260)), (prompt, dict(vts=12))], ids=str)
def test_misaligned(call, bad):
    assert call(**bad) == q.QW3_ERR_ALIGN


def test_no_work_enqueues_nothing():
    assert write(T=0, k=NULL, v=NULL, slots=NULL) == q.QW3_OK
    assert write(pages=0, codes=NULL, scales=NULL) == q.QW3_OK
    assert read(total=0) == q.QW3_OK and read(B=0, table=NULL) == q.QW3_OK
    assert cache(Tq=0) == q.QW3_OK and cache(B=0, Tq=0, cu=NULL) == q.QW3_OK
    assert prompt(B=0) == q.QW3_OK and prompt(Tq=0, qq=NULL) == q.QW3_OK


def test_binding_refuses_before_the_library_is_called():
    """CPU tensors and wrong types, shapes and strides raise in Python."""
    codes, scales = q.new_cache(3, 16, 2, 64, device="cpu")
    assert codes.shape == (3, 2, 2, 16, 64) and codes.dtype is torch.int8 and scales.shape == (3, 2, 2, 16)
    assert q.new_cache(1, 32, 1, 128, torch.float8_e4m3fn, "cpu")[0].dtype is torch.float8_e4m3fn
    for bad in (dict(dtype=torch.uint8), dict(dim=96), dict(page_size=8), dict(page_size=40)):
        with pytest.raises((TypeError, ValueError)):
            q.new_cache(**{**dict(pages=1, page_size=16, heads=2, dim=64, device="cpu"), **bad})
    kv = torch.zeros(4, 2, 64)
    slots = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        q.qcache_write(kv, kv, slots, codes, scales)
    with pytest.raises(TypeError, match="codes"):
        q.qcache_write(kv, kv, slots, codes.view(torch.uint8), scales)
    with pytest.raises(ValueError, match="scales"):
        q.qcache_write(kv, kv, slots, codes, scales[:2])
    b16 = kv.bfloat16()
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        q.qattn_prompt(b16, b16, b16, cu)
    with pytest.raises(TypeError, match="bfloat16"):
        q.qattn_prompt(kv, b16, b16, cu)
    with pytest.raises(ValueError, match="GPU"):
        q.qattn_cache(b16, codes, scales, cu.view(1, 2), cu[:1])
    with pytest.raises(ValueError, match="GPU"):
        q.qcache_read(codes, scales, cu.view(1, 2), cu, 4)


def test_error_status_becomes_an_exception():
    from dequant_gemv_qgemv_amd import _attention
    with pytest.raises(q.Qw3Error) as e:
        _attention._fail(q.QW3_ERR_SHAPE, "qattn_cache")
    assert e.value.status == q.QW3_ERR_SHAPE and "qattn_cache" in str(e.value)
