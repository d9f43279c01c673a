"""CPU checks of the rotary position calls: bad arguments are refused on the
host.  Pointers here are fake and never dereferenced."""
import pytest
import torch

import dequant_gemv_qgemv_amd as q

A = [0x10000 * (i + 1) for i in range(14)]
NULL = None
S = None


def rope(x=A[0], src=0, pos=A[1], rates=A[2], axis=A[3], style=0, out=A[4], T=4, H=2, D=128, R=128, axes=1, ts=256, hs=128):
    return q.raw().qrope(x, src, pos, rates, axis, style, out, T, H, D, R, axes, ts, hs, S)


def write(qq=A[0], k=A[1], v=A[2], src=0, pos=A[3], rates=A[4], axis=A[5], style=0, slots=A[6], qo=A[7], ko=A[8], vo=A[9],
          codes=A[10], scales=A[11], kind=0, T=4, Hq=4, H=2, D=128, R=128, axes=1, pages=8, size=16, qts=512, qhs=128,
          kts=256, khs=128, vts=256, vhs=128):
    return q.raw().qrope_write(qq, k, v, src, pos, rates, axis, style, slots, qo, ko, vo, codes, scales, kind, T, Hq, H, D,
                               R, axes, pages, size, qts, qhs, kts, khs, vts, vhs, S)


SHAPES = [dict(src=2), dict(src=-1), dict(style=2), dict(style=-1), dict(D=96), dict(D=256), dict(R=0), dict(R=8), dict(R=24),
          dict(R=144), dict(D=64, R=80), dict(axes=0), dict(axes=9), dict(H=0), dict(T=-1), dict(T=1 << 24), dict(T=1 << 60)]


@pytest.mark.parametrize("bad", SHAPES + [dict(H=1025), dict(ts=-256), dict(hs=-128), dict(ts=1 << 32), dict(hs=1 << 40)], ids=str)
def test_shapes(bad):
    assert rope(**bad) == q.QW3_ERR_SHAPE


@pytest.mark.parametrize("bad", SHAPES + [
    dict(kind=2), dict(Hq=3), dict(Hq=0), dict(Hq=1026), dict(size=24), dict(size=8), dict(pages=-1), dict(qts=-512),
    dict(kts=1 << 32), dict(vhs=1 << 40)], ids=str)
def test_write_shapes(bad):
    assert write(**bad) == q.QW3_ERR_SHAPE


def test_null_pointers():
    for name in ("x", "pos", "rates", "out"):
        assert rope(**{name: NULL}) == q.QW3_ERR_NULL, name
    for name in ("qq", "k", "v", "pos", "rates", "slots", "qo", "codes", "scales"):
        assert write(**{name: NULL}) == q.QW3_ERR_NULL, name


@pytest.mark.parametrize("call,bad", [
    (rope, dict(x=0x10008)), (rope, dict(out=0x10008)), (rope, dict(pos=0x10002)), (rope, dict(rates=0x10004)),
    (rope, dict(axis=0x10002)), (rope, dict(ts=260)), (rope, dict(src=1, hs=130)),
    (write, dict(qq=0x10008)), (write, dict(k=0x10008)), (write, dict(v=0x10008)), (write, dict(qo=0x10008)),
    (write, dict(ko=0x10008)), (write, dict(vo=0x10008)), (write, dict(codes=0x10008)), (write, dict(scales=0x10008)),
    (write, dict(slots=0x10004)), (write, dict(rates=0x10004)), (write, dict(pos=0x10001)), (write, dict(axis=0x10001)),
    (write, dict(qts=516)), (write, dict(khs=4)), (write, dict(src=1, vts=254))], ids=str)
def test_alignment(call, bad):
    assert call(**bad) == q.QW3_ERR_ALIGN


def test_no_tokens_is_no_work():
    assert rope(T=0, x=NULL, out=NULL) == q.QW3_OK
    assert write(T=0, qq=NULL, codes=NULL) == q.QW3_OK


def test_binding_refuses_the_cpu_and_wrong_types():
    x, p, r = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        q.qrope(x, p, r)
    with pytest.raises(TypeError):
        q.qrope(x.double(), p, r)
    codes, scales = q.new_cache(2, 16, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        q.qrope_write(x, x, x, p, r, torch.zeros(3, dtype=torch.int64), codes, scales)
