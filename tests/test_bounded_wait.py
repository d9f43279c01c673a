"""The bounded wait of the kernels that pass a flag between workgroups (csrc/qw3_units.h),
compiled by g++: it ends whatever the flag does, and says whether it came."""
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dequant_gemv_qgemv_amd", "csrc")

PROGRAM = r"""
#include "qw3_units.h"

int main() {
    for (int polls = 0; polls < 5; ++polls)
        for (int comes = 0; comes < 8; ++comes) {  // the flag is there from look `comes` on; 7: never
            int looks = 0, pauses = 0;
            const bool seen = qw3_units::wait_until([&] { return looks++ >= comes && comes < 7; }, [&] { ++pauses; }, polls);
            if (seen != (comes < 7 && comes < polls)) return 1;
            if (looks > polls || pauses != (seen ? looks - 1 : looks)) return 2;
        }
    return 0;
}
"""


def test_a_wait_ends_and_says_how(tmp_path):
    (tmp_path / "p.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", str(tmp_path / "p"), str(tmp_path / "p.cpp")], check=True)
    assert subprocess.run([str(tmp_path / "p")]).returncode == 0


def test_no_wait_runs_out_in_silence():
    """Every look for another workgroup's flag goes through the bounded wait, whose answer is used."""
    waits = 0
    for name in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, name)).read()
        assert len(re.findall(r"s_sleep", text)) == len(re.findall(r"wait_until\(", text)) - (name == "qw3_units.h"), name
        waits += len(re.findall(r"if \(!wait_until\(", text))
    assert waits == 1
