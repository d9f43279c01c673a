"""Layouts that the kernels rest on, asserted where the compiler sees them: the units'
own declarations, checked on the host."""
import os
import subprocess

import pytest

from dequant_gemv_qgemv_amd import _build

CASES = {
    # read and written as int4 in every element of an array
    "PickSpace": ("qw3_blocks.hip", """
template <int T>
constexpr bool whole = alignof(PickSpace<T>) >= sizeof(int4) && sizeof(PickSpace<T>) % sizeof(int4) == 0 &&
                       offsetof(PickSpace<T>, bins) % sizeof(int4) == 0;
static_assert(whole<64> && whole<256> && whole<1024>, "16-byte pieces of PickSpace");
"""),
}


@pytest.mark.skipif(not os.path.exists(_build.HIPCC), reason="no hipcc")
@pytest.mark.parametrize("name", CASES)
def test_layout(tmp_path, name):
    unit, asserted = CASES[name]
    src = tmp_path / "p.hip"
    src.write_text('#include <stddef.h>\n#include "%s"\n%s' % (unit, asserted))
    r = subprocess.run([_build.HIPCC] + _build.HIP_FLAGS + ["--cuda-host-only", "-fsyntax-only", "-I", _build.CSRC, str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
