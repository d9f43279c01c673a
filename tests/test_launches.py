"""What the library launches, and in which order, on the CPU: a program that loads
libqw3.so defines the runtime's calls itself, so that a launch is a line of its
record and nothing runs.  Pointers are fake and never dereferenced."""
import os
import subprocess

import pytest

import dequant_gemv_qgemv_amd as q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <dlfcn.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <chrono>
#include <condition_variable>
#include <mutex>
#include <thread>
#include <vector>
#include "qw3.h"

struct dim3 { uint32_t x, y, z; };
struct Launch { int who; uint64_t groups; };

static std::mutex m;
static std::condition_variable changed;
static std::vector<Launch> launches;
static thread_local int me = 0;
static bool pause_first = false;  // thread 1 waits behind its first launch until thread 2 has launched, or a while

static thread_local dim3 grid_, block_;
static thread_local size_t lds_;
static thread_local void *stream_;

// the runtime, as far as the library asks for it
extern "C" {
int __hipPushCallConfiguration(dim3 g, dim3 b, size_t lds, void *s) { grid_ = g, block_ = b, lds_ = lds, stream_ = s; return 0; }
int __hipPopCallConfiguration(dim3 *g, dim3 *b, size_t *lds, void **s) { *g = grid_, *b = block_, *lds = lds_, *s = stream_; return 0; }
int hipGetDevice(int *d) { *d = 0; return 0; }
int hipDeviceGetAttribute(int *v, int, int) { *v = 256; return 0; }
int hipGetLastError() { return 0; }
int hipMalloc(void **p, size_t) {
    static uintptr_t next = uintptr_t(1) << 40;
    std::lock_guard<std::mutex> l(m);
    *p = (void *)next, next += uintptr_t(1) << 36;
    return 0;
}
int hipFree(void *) { return 0; }
int hipGetSymbolAddress(void **p, const void *) { *p = (void *)(uintptr_t(1) << 39); return 0; }
int hipStreamIsCapturing(void *, int *s) { *s = 0; return 0; }
int hipStreamGetCaptureInfo(void *, int *s, unsigned long long *id) { *s = 0, *id = 0; return 0; }
int hipOccupancyMaxActiveBlocksPerMultiprocessor(int *n, const void *, int, size_t) { *n = 2; return 0; }
int hipLaunchKernel(const void *, dim3 g, dim3, void **, size_t, void *) {
    std::unique_lock<std::mutex> l(m);
    const bool first = launches.empty();
    launches.push_back({me, (uint64_t)g.x * g.y * g.z});
    changed.notify_all();
    if (pause_first && first)
        changed.wait_for(l, std::chrono::milliseconds(300), [] { return launches.back().who != me; });
    return 0;
}
}

#define FN(name) decltype(&::name) name##_ = (decltype(&::name))dlsym(lib, #name)
template <class T>
T *at(int i) { return (T *)(uintptr_t(0x100000) * (i + 1)); }

int main(int argc, char **argv) {
    void *lib = dlopen(argv[1], RTLD_NOW);
    if (!lib) { fprintf(stderr, "%s\n", dlerror()); return 2; }
    FN(qcache_compact); FN(qblock_select); FN(qattn_cache); FN(qgemm_w3g128_smallM); FN(qgemm_w3g128_smallM_noalloc);
    auto call = [&](const char *what, void *s) -> int {
        if (!strcmp(what, "compact"))
            return qcache_compact_(at<char>(0), at<float>(1), at<int32_t>(2), at<int32_t>(3), at<int32_t>(4), at<uint8_t>(5),
                                   at<int32_t>(6), 1, 100, 1000, 2, 8, 128, 200, 16, s);
        if (!strcmp(what, "select"))
            return qblock_select_(at<uint16_t>(0), at<int8_t>(1), at<float>(2), at<int32_t>(3), at<int32_t>(4), at<int32_t>(5),
                                  at<int32_t>(6), 2, 3000, 6, 8, 2, 128, 6000, 16, 20, 1, 1, 1024, 128, s);
        if (!strcmp(what, "attention"))
            return qattn_cache_(at<uint16_t>(0), at<char>(1), at<float>(2), 0, at<int32_t>(3), at<int32_t>(4), nullptr, nullptr,
                                at<uint16_t>(5), 4, 100, 4, 64, 8, 128, 500, 16, 8192, 128, 0.1f, s);
        const bool fixed = !strncmp(what, "noalloc", 7);
        const int64_t M = atoll(what + (fixed ? 7 : 4));
        return (fixed ? qgemm_w3g128_smallM_noalloc_ : qgemm_w3g128_smallM_)(at<uint16_t>(0), at<int32_t>(1), at<uint16_t>(2),
                                                                            at<float>(3), M, 1024, 8192, s);
    };
    if (!strcmp(argv[2], "select")  && argc > 6) {  // new tokens, sequences, table width, kv heads: the workgroups of each launch
        const int64_t Tq = atoll(argv[3]), B = atoll(argv[4]), width = atoll(argv[5]), H = atoll(argv[6]);
        const int status = qblock_select_(at<uint16_t>(0), at<int8_t>(1), at<float>(2), at<int32_t>(3), at<int32_t>(4),
                                          Tq == B ? nullptr : at<int32_t>(5), at<int32_t>(6), B, width, Tq, H, H, 128, 60000, 16,
                                          20, 1, 1, 128 * H, 128, at<void>(20));
        if (status) { fprintf(stderr, "status %d\n", status); return 3; }
        for (const Launch &x : launches) printf("%llu ", (unsigned long long)x.groups);
        printf("\n");
        fflush(stdout);
        _Exit(0);
    }
    // two threads, the second of which calls once the first is between two of its launches
    pause_first = true;
    int first = 0, second = 0;
    std::thread a([&] { me = 1; first = call(argv[2], at<void>(20)); });
    std::thread b([&] {
        me = 2;
        { std::unique_lock<std::mutex> l(m); changed.wait(l, [] { return !launches.empty(); }); }
        second = call(argv[3], at<void>(20 + atoi(argv[4])));
    });
    a.join(), b.join();
    if (first || second) { fprintf(stderr, "status %d %d\n", first, second); return 3; }
    for (const Launch &x : launches) printf("%d ", x.who);
    printf("\n");
    fflush(stdout);
    _Exit(0);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("launches")
    (d / "p.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-rdynamic", "-I", os.path.join(ROOT, "include"), "-o", str(d / "p"),
                    str(d / "p.cpp"), "-ldl", "-pthread"], check=True)

    def run(*args):
        r = subprocess.run([str(d / "p"), q.library_path()] + [str(a) for a in args], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        return r.stdout.split()
    return run


SEVERAL = ["compact", "select", "gemm16", "gemm60", "gemm512"]  # calls of several launches that pass data in the stream's buffer


@pytest.mark.parametrize("second", SEVERAL + ["attention"])
@pytest.mark.parametrize("first", SEVERAL)
def test_calls_of_two_threads_on_one_stream_do_not_mix(program, first, second):
    order = program(first, second, 0)
    n = order.count("1")
    assert n > 1 and len(order) > n and order == ["1"] * n + ["2"] * (len(order) - n)


@pytest.mark.parametrize("first,second", [("noalloc16", "noalloc512"), ("noalloc512", "noalloc60")])
def test_calls_of_two_threads_in_the_static_array_do_not_mix(program, first, second):
    order = program(first, second, 0)
    n = order.count("1")
    assert n > 1 and len(order) > n and order == ["1"] * n + ["2"] * (len(order) - n)


@pytest.mark.parametrize("first,second", [("compact", "select"), ("select", "attention"), ("gemm16", "gemm16")])
def test_calls_on_two_streams_do_not_wait_for_each_other(program, first, second):
    assert program(first, second, 1)[:2] == ["1", "2"]


@pytest.mark.parametrize("rows,batch,width,heads", [(30000, 1, 8192, 8), (30000, 7500, 8192, 8), (30000, 30000, 8192, 8),
                                                    (60000, 3, 60000, 16), (5000, 5000, 300, 1), (90, 1, 1 << 20, 64)])
def test_the_work_of_a_selection_grows_with_its_rows(program, rows, batch, width, heads):
    """However many batches the scores are made in: tiles of 16 rows, one more for each sequence that a batch has rows of,
    each with up to 64 workgroups for its pages; and one workgroup for each row to pick."""
    groups = [int(x) for x in program("select", rows, batch, width, heads)]
    batches = max(len(groups) // 2, 1)
    some = min(-(-width // 256), 64)
    tiles = rows // 16 + min(batch * batches, rows) + batches
    assert sum(groups) <= heads * (some * tiles + rows)
