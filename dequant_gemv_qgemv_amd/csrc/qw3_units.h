// How the attention calls count their work: which rows a sequence has, what an
// item is worth in units, which run of units a workgroup takes; and a wait that
// ends.  Constexpr functions alone, without HIP, so that a test runs these very
// ones on the CPU over what no kernel should meet unprepared.
#pragma once

#include <stdint.h>

namespace qw3_units {

constexpr int larger(int a, int b) { return a > b ? a : b; }
constexpr int smaller(int a, int b) { return a < b ? a : b; }

// A start as a row number, whatever the array holds.
constexpr int clamp_row(int x, int total) { return smaller(larger(x, 0), total); }

// The rows of a sequence that the starts give begin .. end - 1 of `total`.
// `floor`: the largest start before it (clamped, 0 for the first).  A start below
// an earlier one counts as that one, so no row belongs to two sequences and all
// sequences together have at most `total` rows, which the host's bound on the
// work of a call and the kernels' 32-bit sums rest on.
struct Rows {
    int first, n;
};
constexpr Rows rows_of(int begin, int end, int floor, int total) {
    const int first = larger(clamp_row(begin, total), floor);
    return Rows{first, larger(clamp_row(end, total) - first, 0)};
}

// qattn_cache: an item is (sequence, kv head, block of R query rows); its work is
// counted in units: kSetup for beginning and ending it, and one for each
// unit_of(R) keys (with few rows 32 for each of a workgroup's 4 waves, with many
// a tile that the waves share), at least one, so that an empty cache still writes
// its zeros.
constexpr int unit_of(int R) { return R <= 32 ? 128 : 64; }
constexpr int kSetup = 2;
constexpr int units_of_item(int len, int R) { return kSetup + larger((len + unit_of(R) - 1) / unit_of(R), 1); }
constexpr int blocks_of(int rows, int R) { return (rows + R - 1) / R; }

// Whether the units of a call fit 31 bits whatever its starts and lengths, from
// what the host knows: rows Tq and query heads a kv head G, sequences B, kv heads
// H and the most keys that a table can name.
constexpr bool units_fit(int64_t Tq, int64_t G, int64_t B, int64_t H, int64_t keys, int R) {
    const int64_t most = (keys + 2 * unit_of(R) - 1) / unit_of(R) + kSetup;
    const int64_t items = (Tq * G / R + B) * H;
    return most <= 0x7fffffff / (items + 1);
}

// The run of workgroup `group` of `groups` over `total` units: equal runs, no
// shorter than `least`.
struct Run {
    int per, begin, end;
};
constexpr Run run_of(int total, int groups, int least, int group) {
    const int per = larger(larger((int)(((uint32_t)total + (uint32_t)groups - 1) / (uint32_t)groups), least), 1);
    const int64_t at = (int64_t)group * per;
    const int begin = at < total ? (int)at : total;
    return Run{per, begin, begin + smaller(per, total - begin)};
}
// The workgroup whose run holds a unit.
constexpr int group_of(int unit, int per) { return (int)((uint32_t)unit / (uint32_t)per); }

// The counters of a stream: four banks of kCounts.  A call counts in one bank and
// clears the other of its pair for the call behind it, which runs later: what a
// bank holds from before, whatever that is, lasts for no more than one call.
// Calls that a graph captures have a pair of their own, cleared by a launch of its
// own (`fresh`) before the first of a capture: a replay starts from zeros, however
// the one before it ended, and leaves the eager calls' banks alone.  That launch
// costs a replay 4 us, once whatever the number of its calls (80 decodes of one
// token: 664 -> 674 us).  Counts are set
// back to zero by the call itself too, so the order in which threads enqueue on one
// stream does not matter.
constexpr int kCounts = 1024;
struct BankChoice {
    int use, clear;
    bool fresh;
};
struct Banks {
    int eager = 0, captured = 2;
    unsigned long long capture = 0;  // the last capture's id
    bool captures = false;           // there was one
    constexpr BankChoice choose(bool capturing, unsigned long long id) {
        if (!capturing) {
            const int use = eager;
            eager = 1 - use;
            return BankChoice{use, eager, false};
        }
        const bool fresh = !captures || capture != id;
        const int use = fresh ? 2 : captured;
        captures = true, capture = id, captured = 5 - use;
        return BankChoice{use, captured, fresh};
    }
};

// A wait that ends: looks until seen(), `polls` times at most, with pause() after each look
// in vain.  Whether it was seen.
template <class Seen, class Pause>
constexpr bool wait_until(Seen seen, Pause pause, int polls) {
    for (int i = 0; i < polls; ++i) {
        if (seen()) return true;
        pause();
    }
    return false;
}

}  // namespace qw3_units
