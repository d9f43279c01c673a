"""CPU checks of the calls that attend over selected pages: bad arguments are
refused on the host.  Pointers here are fake and never dereferenced."""
import pytest
import torch

import dequant_gemv_qgemv_amd as q

A = [0x10000 * (i + 1) for i in range(10)]
NULL = None
S = None


def bounds(codes=A[0], scales=A[1], kind=0, table=A[2], lens=A[3], cu=A[4], out=A[5], steps=A[6], B=2, maxp=4, Tq=6, H=2, D=128,
           pages=8, size=16):
    return q.raw().qcache_bounds(codes, scales, kind, table, lens, cu, out, steps, B, maxp, Tq, H, D, pages, size, S)


def select(qq=A[0], limits=A[1], steps=A[2], table=A[3], lens=A[4], cu=A[5], picks=A[6], B=2, maxp=4, Tq=6, Hq=8, H=2, D=128,
           pages=8, size=16, count=3, first=1, recent=1, ts=1024, hs=128):
    return q.raw().qblock_select(qq, limits, steps, table, lens, cu, picks, B, maxp, Tq, Hq, H, D, pages, size, count, first,
                                 recent, ts, hs, S)


def attend(qq=A[0], codes=A[1], scales=A[2], kind=0, table=A[3], lens=A[4], cu=A[5], picks=A[6], out=A[7], B=2, maxp=4, Tq=6,
           Hq=8, H=2, D=128, pages=8, size=16, count=3, ts=1024, hs=128, sm=0.1):
    return q.raw().qattn_blocks(qq, codes, scales, kind, table, lens, cu, picks, out, B, maxp, Tq, Hq, H, D, pages, size, count,
                                ts, hs, sm, S)


SHAPES = [dict(H=0), dict(H=1 << 20), dict(D=96), dict(D=256), dict(size=8), dict(size=48), dict(size=131072), dict(pages=-1),
          dict(B=-1), dict(B=1 << 20), dict(Tq=-1), dict(Tq=1 << 27), dict(maxp=-1), dict(maxp=1 << 27), dict(maxp=1 << 60), dict(cu=NULL)]


@pytest.mark.parametrize("bad", SHAPES, ids=str)
@pytest.mark.parametrize("call", [bounds, select, attend])
def test_sequences(call, bad):
    assert call(**bad) == q.QW3_ERR_SHAPE


PICKS = [dict(Hq=7), dict(Hq=0), dict(Hq=1026), dict(count=0), dict(count=-1), dict(count=65537), dict(ts=-8), dict(hs=-8),
         dict(ts=1 << 32), dict(hs=1 << 40), dict(Tq=1 << 26, H=2, Hq=8)]


@pytest.mark.parametrize("call,bad", [(c, b) for c in (select, attend) for b in PICKS] + [
    (bounds, dict(kind=2)), (bounds, dict(kind=-1)), (bounds, dict(B=65536, H=1024, Tq=1 << 20)), (attend, dict(kind=2)),
    (attend, dict(sm=0.0)), (attend, dict(sm=-1.0)), (attend, dict(sm=float("inf"))), (attend, dict(sm=float("nan"))),
    (attend, dict(count=65536, size=32768)), (attend, dict(Tq=1 << 20, H=64, Hq=64)), (select, dict(first=-1)),
    (select, dict(recent=0)), (select, dict(first=2, recent=2)), (select, dict(first=4)), (select, dict(recent=1 << 62, first=1)),
    (select, dict(Tq=1 << 21))], ids=str)
def test_shapes(call, bad):
    assert call(**bad) == q.QW3_ERR_SHAPE


@pytest.mark.parametrize("call,names", [
    (bounds, ("codes", "scales", "table", "lens", "out", "steps")), (select, ("qq", "limits", "steps", "table", "lens", "picks")),
    (attend, ("qq", "codes", "scales", "table", "lens", "picks", "out"))])
def test_null_pointers(call, names):
    for name in names:
        assert call(**{name: NULL}) == q.QW3_ERR_NULL, name


@pytest.mark.parametrize("call,bad", [
    (bounds, dict(codes=0x10008)), (bounds, dict(scales=0x10008)), (bounds, dict(table=0x10002)), (bounds, dict(lens=0x10002)),
    (bounds, dict(cu=0x10002)), (bounds, dict(out=0x10008)), (bounds, dict(steps=0x10002)),
    (select, dict(qq=0x10008)), (select, dict(limits=0x10008)), (select, dict(steps=0x10002)), (select, dict(table=0x10002)),
    (select, dict(lens=0x10001)), (select, dict(cu=0x10001)), (select, dict(picks=0x10002)), (select, dict(ts=1028)),
    (select, dict(hs=4)), (attend, dict(qq=0x10008)), (attend, dict(codes=0x10008)), (attend, dict(scales=0x10008)),
    (attend, dict(table=0x10002)), (attend, dict(lens=0x10001)), (attend, dict(cu=0x10001)), (attend, dict(picks=0x10002)),
    (attend, dict(out=0x10008)), (attend, dict(ts=1028)), (attend, dict(hs=4))], ids=str)
def test_alignment(call, bad):
    assert call(**bad) == q.QW3_ERR_ALIGN


def test_nothing_to_do():
    assert bounds(B=0, Tq=0, codes=NULL) == q.QW3_OK
    assert bounds(Tq=0, codes=NULL) == q.QW3_OK
    assert select(B=0, Tq=0, qq=NULL) == q.QW3_OK
    assert attend(Tq=0, qq=NULL, out=NULL) == q.QW3_OK


def test_binding_refuses_the_cpu_and_wrong_types():
    codes, scales = q.new_cache(4, 16, 2, 64, device="cpu")
    limits, steps = q.new_bounds(codes)
    assert limits.shape == (4, 2, 2, 64) and steps.shape == (4, 2)
    table, lens = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    x = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.qcache_bounds(codes, scales, table, lens, limits, steps)
    with pytest.raises(ValueError):
        q.qblock_select(x, limits, steps, table, lens, 2, 16)
    with pytest.raises(TypeError):
        q.qblock_select(x.float(), limits, steps, table, lens, 2, 16)
    with pytest.raises(ValueError):
        q.qattn_blocks(x, codes, scales, table, lens, torch.zeros(3, 2, 2, dtype=torch.int32))
