"""CPU checks of the cache and attention calls' limits as the header states them.
Pointers are fake and never dereferenced: a call inside its limits here is stopped
by a misaligned pointer, which is looked at after the sizes."""
import pytest

import dequant_gemv_qgemv_amd as q
from test_attention_abi import cache, prompt, read, write

TOKENS = 1 << 26


@pytest.mark.parametrize("bad", [dict(kts=-256), dict(khs=-128), dict(vts=-256), dict(vhs=-8), dict(kts=1 << 32),
                                 dict(vts=1 << 62), dict(khs=1 << 40), dict(src=1, kts=-4)], ids=str)
def test_write_refuses_strides(bad):
    """A negative one would read before its array."""
    assert write(**bad) == q.QW3_ERR_SHAPE


@pytest.mark.parametrize("call,bad,good", [
    (write, dict(T=TOKENS + 1, H=1), dict(T=TOKENS, H=1)),
    (write, dict(T=1 << 26, H=8), dict(T=(1 << 26) - 32, H=7)),          # 2^29 rows of 128 channels
    (write, dict(T=1 << 26, H=16, D=64), dict(T=1 << 26, H=15, D=64)),   # 2^30 of 64
    (read, dict(total=TOKENS + 1), dict(total=TOKENS)),
    (cache, dict(Tq=TOKENS + 1, Hq=1, H=1), dict(Tq=TOKENS, Hq=2, H=2)),
    (prompt, dict(Tq=TOKENS + 1), dict(Tq=TOKENS)),
    (prompt, dict(B=65536, Hq=256, H=1), dict(B=65536, Hq=128, H=1)),
    (prompt, dict(Tq=TOKENS, Hq=32), dict(Tq=TOKENS, Hq=24)),
], ids=str)
def test_sizes(call, bad, good):
    assert call(**bad) == q.QW3_ERR_SHAPE
    pointer = {write: "k", read: "k", cache: "qq", prompt: "qq"}[call]
    assert call(**{**good, pointer: 0x10008}) == q.QW3_ERR_ALIGN


def test_strides_inside_the_limits():
    assert write(kts=(1 << 32) - 8, khs=(1 << 40) - 8, k=0x10008) == q.QW3_ERR_ALIGN
    assert prompt(kts=(1 << 23) - 8, khs=(1 << 40) - 8, qq=0x10008) == q.QW3_ERR_ALIGN
