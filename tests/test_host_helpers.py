"""Host helpers of the library that need no HIP (csrc/qw3_host.h), compiled by g++."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dequant_gemv_qgemv_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <new>
#include <vector>
#include "qw3_host.h"

static int left;  // allocations that still succeed
template <class T>
struct Scarce {
    using value_type = T;
    Scarce() = default;
    template <class U> Scarce(const Scarce<U> &) {}
    T *allocate(std::size_t n) {
        if (left-- <= 0) throw std::bad_alloc();
        return static_cast<T *>(::operator new(n * sizeof(T)));
    }
    void deallocate(T *p, std::size_t) { ::operator delete(p); }
    bool operator==(const Scarce &) const { return true; }
    bool operator!=(const Scarce &) const { return false; }
};

int main() {
    std::vector<int, Scarce<int>> v;
    left = 0;
    if (qw3_host::room_for_one(v)) return 1;
    left = 2;
    int pushed = 0;
    while (pushed < 1000 && qw3_host::room_for_one(v)) {
        left -= 100;  // push_back itself must not allocate
        v.push_back(pushed++);
        left += 100;
    }
    if (pushed < 4 || pushed == 1000) return 2;  // stopped by memory, not by an exception
    for (int i = 0; i < pushed; ++i)
        if (v[i] != i) return 3;
    left = 1;
    return qw3_host::room_for_one(v) ? 0 : 4;
}
"""


def test_tables_that_cannot_grow_say_so(tmp_path):
    """An allocation that fails becomes a status, no exception."""
    (tmp_path / "p.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", str(tmp_path / "p"), str(tmp_path / "p.cpp")],
                   check=True)
    assert subprocess.run([str(tmp_path / "p")]).returncode == 0


def test_every_table_of_the_library_asks_for_room():
    """Each push_back stands behind a question for room in the same function."""
    for name in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, name)).read()
        for at in range(text.count(".push_back(")):
            end = [i for i in range(len(text)) if text.startswith(".push_back(", i)][at]
            table = text[:end].split()[-1].split("(")[-1]
            assert "room_for_one(%s)" % table in text[max(0, end - 1500):end], (name, table)
