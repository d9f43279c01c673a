"""CPU checks of the calls on the cache's pages: bad arguments are refused on the
host.  Pointers here are fake and never dereferenced."""
import pytest
import torch

import dequant_gemv_qgemv_amd as q

A = [0x10000 * (i + 1) for i in range(10)]
NULL = None
S = None


def reserve(refs=A[0], table=A[1], lens=A[2], cu=A[3], slots=A[4], out=A[5], copies=A[6], B=2, maxp=4, total=5, pages=8, size=16):
    return q.raw().qcache_reserve(refs, table, lens, cu, slots, out, copies, B, maxp, total, pages, size, S)


def fork(refs=A[0], table=A[1], lens=A[2], parents=A[3], to=A[4], out=A[5], B=2, Bo=3, maxp=4, pages=8, size=16):
    return q.raw().qcache_fork(refs, table, lens, parents, to, out, B, Bo, maxp, pages, size, S)


def copy(codes=A[0], scales=A[1], copies=A[2], n=2, layers=3, H=2, D=128, pages=8, size=16):
    return q.raw().qcache_copy(codes, scales, copies, n, layers, H, D, pages, size, S)


def compact(codes=A[0], scales=A[1], table=A[2], lens=A[3], cu=A[4], keep=A[5], out=A[6], B=2, maxp=4, Tq=5, layers=3, H=2,
            D=128, pages=8, size=16):
    return q.raw().qcache_compact(codes, scales, table, lens, cu, keep, out, B, maxp, Tq, layers, H, D, pages, size, S)


TABLES = [dict(B=-1), dict(B=1 << 20), dict(maxp=-1), dict(maxp=1 << 27), dict(maxp=1 << 60), dict(B=60000, maxp=1 << 20),
          dict(size=8), dict(size=48), dict(size=1 << 17), dict(pages=-1), dict(pages=1 << 31)]


@pytest.mark.parametrize("bad", TABLES, ids=str)
@pytest.mark.parametrize("call", [reserve, fork, compact])
def test_tables(call, bad):
    assert call(**bad) == q.QW3_ERR_SHAPE


@pytest.mark.parametrize("call,bad", [
    (reserve, dict(total=-1)), (reserve, dict(total=1 << 27)), (reserve, dict(cu=NULL)),
    (fork, dict(Bo=-1)), (fork, dict(Bo=1 << 20)), (fork, dict(Bo=60000, maxp=1 << 20)),
    (copy, dict(n=-1)), (copy, dict(n=1 << 27)), (copy, dict(layers=-1)), (copy, dict(layers=1025)), (copy, dict(H=0)),
    (copy, dict(D=96)), (copy, dict(size=20)), (copy, dict(n=1 << 24)), (copy, dict(n=1 << 20, layers=1000)),
    (compact, dict(Tq=-1)), (compact, dict(Tq=1 << 27)), (compact, dict(cu=NULL)), (compact, dict(layers=0)),
    (compact, dict(layers=1025)), (compact, dict(D=32)), (compact, dict(H=1025)), (compact, dict(B=60000, H=300, layers=2)), (compact, dict(Tq=1 << 26, H=16)), (compact, dict(Tq=1 << 26, H=9))], ids=str)
def test_shapes(call, bad):
    assert call(**bad) == q.QW3_ERR_SHAPE


@pytest.mark.parametrize("call,names", [
    (reserve, ("refs", "table", "lens", "slots", "out", "copies")), (fork, ("refs", "table", "lens", "parents", "to", "out")),
    (copy, ("codes", "scales", "copies")), (compact, ("codes", "scales", "table", "lens", "keep", "out"))])
def test_null_pointers(call, names):
    for name in names:
        assert call(**{name: NULL}) == q.QW3_ERR_NULL, name


@pytest.mark.parametrize("call,bad", [
    (reserve, dict(refs=0x10008)), (reserve, dict(table=0x10002)), (reserve, dict(lens=0x10002)), (reserve, dict(cu=0x10001)),
    (reserve, dict(slots=0x10004)), (reserve, dict(out=0x10002)), (reserve, dict(copies=0x10004)),
    (fork, dict(refs=0x10004)), (fork, dict(table=0x10002)), (fork, dict(lens=0x10002)), (fork, dict(parents=0x10002)),
    (fork, dict(to=0x10002)), (fork, dict(out=0x10002)),
    (copy, dict(codes=0x10008)), (copy, dict(scales=0x10008)), (copy, dict(copies=0x10004)),
    (compact, dict(codes=0x10008)), (compact, dict(scales=0x10008)), (compact, dict(table=0x10002)), (compact, dict(lens=0x10002)),
    (compact, dict(cu=0x10002)), (compact, dict(out=0x10002))], ids=str)
def test_alignment(call, bad):
    assert call(**bad) == q.QW3_ERR_ALIGN


def test_nothing_to_do():
    assert reserve(B=0, total=0, lens=NULL, table=NULL) == q.QW3_OK
    assert fork(B=0, Bo=0, refs=NULL) == q.QW3_OK
    assert copy(n=0, codes=NULL) == q.QW3_OK
    assert copy(layers=0, codes=NULL) == q.QW3_OK
    assert compact(B=0, Tq=0, codes=NULL, lens=NULL) == q.QW3_OK


def test_binding_refuses_the_cpu_and_wrong_types():
    refs, table, lens = torch.zeros(8, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    codes, scales = q.new_cache(8, 16, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        q.qcache_reserve(refs, table, lens, 16)
    with pytest.raises(ValueError):
        q.qcache_fork(refs, table, lens, lens, 16)
    with pytest.raises(ValueError):
        q.qcache_copy(codes, scales, table[:, :2])
    with pytest.raises(TypeError):
        q.qcache_copy(codes.view(torch.uint8), scales, table[:, :2])
    with pytest.raises(ValueError):
        q.qcache_compact(codes, scales, table, lens, torch.zeros(2, dtype=torch.bool))
    with pytest.raises(ValueError):
        q.qcache_compact(codes[0], scales, table, lens, torch.zeros(2, dtype=torch.bool))
