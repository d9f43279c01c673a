"""The accounting of the attention calls (csrc/qw3_units.h) on the CPU: whatever
the starts and lengths hold, the units of a call stay inside the host's bound and
every item is finished by workgroups that exist, each counted once.  The functions
are the kernels' own, compiled by g++; the walk over a workgroup's run is written
here from their description."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dequant_gemv_qgemv_amd", "csrc")

SHIM = r"""
#include <vector>
#include <map>
#include <cmath>
#include "qw3_units.h"
using namespace qw3_units;

// 0: as it should be; out[0] the units of the call, out[1] the rows of all sequences
extern "C" int walk(const int *cu, const int *lens, int B, int Tq, int G, int H, int keys, int R, int groups,
                    double join, int64_t *out) {
    std::vector<Rows> rows(B);
    std::vector<int> per_item(B);
    int64_t total = 0, all_rows = 0;
    int floor = 0, longest = 0;
    for (int b = 0; b < B; ++b) {
        rows[b] = rows_of(cu[b], cu[b + 1], floor, Tq);
        if (rows[b].first < 0 || rows[b].n < 0 || rows[b].first + (int64_t)rows[b].n > Tq) return 1;
        if (rows[b].first < floor) return 2;  // a row of an earlier sequence
        floor = larger(floor, clamp_row(cu[b], Tq));
        if (floor != rows[b].first) return 3;
        per_item[b] = units_of_item(larger(0, smaller(lens[b], keys)), R);
        all_rows += rows[b].n;
        total += (int64_t)per_item[b] * blocks_of(rows[b].n * G, R) * H;
        if (rows[b].n) longest = larger(longest, per_item[b]);
    }
    out[0] = total, out[1] = all_rows;
    if (!units_fit(Tq, G, B, H, keys, R)) return 0;  // refused on the host
    if (total > 0x7fffffff) return 4;
    if (groups == 0) return 0;
    const int least = (int)std::sqrt((float)join * (float)longest);
    // who works on which item, and whom the item expects
    std::vector<int64_t> start(1, 0);
    for (int b = 0; b < B; ++b) start.push_back(start[b] + (int64_t)per_item[b] * blocks_of(rows[b].n * G, R) * H);
    std::map<int64_t, std::pair<int, int>> expects;  // item's first unit -> first and last workgroup
    std::map<int64_t, std::vector<int>> came;
    int64_t covered = 0;
    for (int g = 0; g < groups; ++g) {
        const Run run = run_of((int)total, groups, least, g);
        if (run.begin < 0 || run.end < run.begin || run.end > total || run.per < 1) return 5;
        covered += run.end - run.begin;
        int u = run.begin, b = 0, shared = 0;
        while (u < run.end) {
            while (u >= start[b + 1]) ++b;
            const int64_t begin = start[b] + (u - start[b]) / per_item[b] * per_item[b];
            if (u < begin + kSetup) u = (int)(begin + kSetup);
            const int count = smaller((int)(begin + per_item[b]), run.end) - u;
            if (count <= 0) break;
            const int first = group_of((int)begin + kSetup, run.per), last = group_of((int)begin + per_item[b] - 1, run.per);
            if (first > last || first > g || last < g || last >= groups) return 6;
            if (first != last && ++shared > 2) return 7;
            expects[begin] = {first, last};
            came[begin].push_back(g);
            u += count;
        }
    }
    if (covered != total) return 8;
    for (const auto &e : expects)
        if ((int)came[e.first].size() != e.second.second - e.second.first + 1) return 9;
    int64_t items = 0;
    for (int b = 0; b < B; ++b) items += (int64_t)blocks_of(rows[b].n * G, R) * H;
    return (int64_t)expects.size() == items ? 0 : 10;
}

extern "C" void *banks_new() { return new Banks(); }
extern "C" void banks_delete(void *b) { delete static_cast<Banks *>(b); }
extern "C" void banks_choose(void *b, int capturing, unsigned long long id, int *out) {
    const BankChoice c = static_cast<Banks *>(b)->choose(capturing != 0, id);
    out[0] = c.use, out[1] = c.clear, out[2] = c.fresh;
}
"""


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    d = tmp_path_factory.mktemp("units")
    src, lib = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, "-o", str(lib), str(src)],
                   check=True)
    return ctypes.CDLL(str(lib))


@pytest.fixture(scope="module")
def walk(shim):
    fn = shim.walk
    p = np.ctypeslib.ndpointer

    def call(cu, lens, Tq, G, H, keys, R, groups=512, join=0.14):
        cu, lens = np.asarray(cu, np.int32), np.asarray(lens, np.int32)
        out = np.zeros(2, np.int64)
        fn.argtypes = [p(np.int32), p(np.int32)] + [ctypes.c_int] * 7 + [ctypes.c_double, p(np.int64)]
        return fn(cu, lens, len(lens), Tq, G, H, keys, R, groups, join, out), int(out[0]), int(out[1])
    return call


@pytest.mark.parametrize("R", [16, 32, 128, 256])
def test_overlapping_starts_stay_inside_the_bound(walk, R):
    """0, Tq, 0, Tq, ...: counted one by one the sequences would have 9.1e9 units in blocks of 16 rows, which wrap to
    554065408 in 32 bits and leave an item to a workgroup past the last."""
    n = 6000
    cu = np.zeros(n + 1, np.int32)
    cu[1::2] = n
    status, total, rows = walk(cu, [16000] * n, n, 8, 8, 16000, R)
    assert status == 0 and rows == n
    assert total == (2 + -(-16000 // (128 if R <= 32 else 64))) * -(-n * 8 // R) * 8


@pytest.mark.parametrize("seed", range(40))
def test_any_starts_and_lengths(walk, seed):
    rng = np.random.default_rng(seed)
    b = int(rng.integers(1, 200))
    tq = int(rng.integers(1, 500))
    span = 2 ** 31 - 1 if seed % 3 == 0 else tq + 20
    cu = rng.integers(-span - 1, span, b + 1)
    if seed % 3 == 1:
        cu = np.sort(cu)
    lens = rng.integers(-5, 3000, b)
    lens[rng.integers(0, b)] = 2 ** 31 - 1
    for R in (16, 32, 128, 256):
        for groups in (1, 7, 256, 512):
            status, total, rows = walk(cu, lens, tq, int(rng.integers(1, 9)), int(rng.integers(1, 9)), 4096, R, groups,
                                       0.14 if R <= 32 else 0.8)
            assert status == 0 and rows <= tq


def test_starts_that_rise_are_taken_as_they_are(walk):
    status, total, rows = walk([0, 3, 3, 10], [5, 5, 5], 10, 1, 1, 4096, 16)
    assert status == 0 and rows == 10 and total == 3 + 3  # the empty one has no items


def test_the_largest_totals(walk):
    """Near 2^31 units the sums of a run's bounds stay in range."""
    # one kv head, 2^26 rows of one query head over 64 keys: 2^22 blocks of 16 rows
    for lens in ([64], [2 ** 30]):
        status, _, _ = walk([0, 1 << 26], lens, 1 << 26, 1, 1, lens[0], 256, 0)
        assert status == 0
    # the host's bound just holds: 255 sequences of one row, 2^29 keys each, blocks of 256
    status, total, rows = walk(np.arange(256), [(1 << 29) - 300] * 255, 255, 1, 1, (1 << 29) - 300, 256, 512, 0.8)
    assert status == 0 and total > 2 ** 31 - 2 ** 24


# --------------------------------------------------------------- counters ---
class Chooser:
    """The banks of one stream, by the library's own choice."""

    def __init__(self, lib):
        lib.banks_new.restype = ctypes.c_void_p
        self.lib, self.at = lib, ctypes.c_void_p(lib.banks_new())

    def __call__(self, capture=None):
        out = (ctypes.c_int * 3)()
        self.lib.banks_choose(self.at, capture is not None, ctypes.c_ulonglong(capture or 0), out)
        return tuple(out)


class OneBank:
    """One bank for all, set back to zero by whoever is last and by nobody else."""

    def __call__(self, capture=None):
        return 0, None, 0


ITEMS = 4


def run_calls(memory, calls, rng):
    """Runs calls at the same time: each a choice of banks and its items' numbers of parts, its steps taken in turn at
    random; a joined item's count is set back a step later. Returns, for each call, how many of its items were joined
    when all their parts were there, and how many joins came too early."""
    done = [[0, 0] for _ in calls]
    queues, arrived = [], [[0] * ITEMS for _ in calls]
    for (_, _, fresh), parts in calls:
        work = [("count", item) for item, n in enumerate(parts) for _ in range(n)] + [("clear", 0)]
        queues.append([("fresh", 0)] * fresh + [work[i] for i in rng.permutation(len(work))])
    while any(queues):
        n = rng.choice([i for i, s in enumerate(queues) if s])
        (use, clear, _), parts = calls[n]
        step, item = queues[n].pop(0)
        if step == "fresh":
            memory[2][:] = memory[3][:] = [0] * ITEMS
        elif step == "clear" and clear is not None:
            memory[clear][:] = [0] * ITEMS
        elif step == "reset":
            memory[use][item] = 0
        elif step == "count":
            arrived[n][item] += 1
            memory[use][item] += 1
            if memory[use][item] == parts[item]:
                done[n][0 if arrived[n][item] == parts[item] else 1] += 1
                queues[n].insert(0, ("reset", item))
    return done


def counts_after_a_race(chooser, seed):
    """Two graphs captured on one stream, replayed at once with each other and with an eager call; then everything in
    order. Returns how many of the ordered calls joined every item once and in time, of how many."""
    rng = np.random.default_rng(seed)
    memory = [[0] * ITEMS for _ in range(4)]
    parts = lambda: [int(x) for x in rng.integers(1, 6, ITEMS)]  # noqa: E731
    alone = lambda call: run_calls(memory, [call], rng)[0] == [ITEMS, 0]  # noqa: E731
    assert alone((chooser(), parts()))
    graphs = [[(chooser(capture=c), parts()) for _ in range(rng.integers(1, 4))] for c in (7, 8)]
    assert alone((chooser(), parts()))
    for _ in range(3):  # the race: a call of each at a time
        run_calls(memory, [g[rng.integers(0, len(g))] for g in graphs], rng)
    run_calls(memory, [graphs[0][0], (chooser(), parts())], rng)
    good = total = 0
    for _ in range(4):
        for call in [None] + graphs[rng.integers(0, 2)] + [None, None]:
            good, total = good + alone(call or (chooser(), parts())), total + 1
    return good, total


def test_counters_survive_calls_that_overlapped(shim):
    """Calls that share a stream's counters must not overlap; if they do all the same, later ones are right again."""
    for seed in range(60):
        good, total = counts_after_a_race(Chooser(shim), seed)
        assert good == total, seed


def test_the_model_sees_counters_that_stay_damaged():
    spoiled = sum(good != total for good, total in (counts_after_a_race(OneBank(), seed) for seed in range(60)))
    assert spoiled > 30


def test_banks_in_order(shim):
    choose = Chooser(shim)
    assert choose() == (0, 1, 0) and choose() == (1, 0, 0) and choose() == (0, 1, 0)
    assert choose(capture=0) == (2, 3, 1) and choose(capture=0) == (3, 2, 0) and choose(capture=0) == (2, 3, 0)
    assert choose() == (1, 0, 0)
    assert choose(capture=5) == (2, 3, 1) and choose() == (0, 1, 0) and choose(capture=5) == (3, 2, 0)
