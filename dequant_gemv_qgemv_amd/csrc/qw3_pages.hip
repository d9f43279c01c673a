// The pages of the key/value cache: room for new tokens (qcache_reserve), rows of a
// block table that follow others (qcache_fork), whole pages copied (qcache_copy) and
// tokens dropped in place (qcache_compact).  C ABI in include/qw3.h.
//
// Who holds a page is counted: refs[p] is the number of entries of the block table
// that name p, 0 a free page.  All results are whole numbers and moved bytes, and
// do not depend on the order in which workgroups run.
#include "qw3_common.h"
#include "qw3_units.h"

using namespace qw3_shared;
using qw3_units::clamp_row;
using qw3_units::wait_until;

namespace {

// Exclusive prefix sum over the workgroup's kThreads threads; *total: of all.
template <int kThreads>
__device__ __forceinline__ int group_scan(int x, int *total) {
    constexpr int kWaves = kThreads / 64;
    __shared__ int sums[kWaves];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int upto = wave_scan(x);
    __syncthreads();  // the sums of the call before are read
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const int s = sums[w];
        before += w < wave ? s : 0;
        all += s;
    }
    *total = all;
    return before + upto - x;
}

// Inclusive prefix maximum over the workgroup, of values >= 0.
template <int kThreads>
__device__ __forceinline__ int group_scan_max(int x) {
    constexpr int kWaves = kThreads / 64;
    __shared__ int tops[kWaves];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    x = wave_scan_max(x);
    __syncthreads();
    if (lane == 63) tops[wave] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) x = w < wave ? max(x, tops[w]) : x;
    return x;
}

// ---------------------------------------------------------------- reserve --
struct ReserveArgs {
    int32_t *refs, *table;
    const int32_t *lens, *cu;
    int64_t *slots;
    int32_t *lens_out, *copies;
    int B, total, shift;
    int64_t max_pages, pages;
};

constexpr int kWide = 1024;

// Of what is sorted in ascending order the last place whose value is at most x.
__device__ __forceinline__ int last_at_most(const int *v, int n, int x) {
    int lo = 0, hi = n;  // v[lo] <= x < v[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (v[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// One workgroup: the work is small (one entry of the table for each page that new
// tokens reach) and each step needs the whole of the one before, so more workgroups
// would cost launches.  A thread has a sequence, then an entry, then 16 pages, then
// a need, then a token:
//   1  the needs, in order of sequence and entry, are listed in `slots`: an entry's
//      number in the table (32 bits).  There are at most as many as tokens, since
//      each page in a sequence's range takes one of its tokens;
//   2  the free pages are counted through in order, the k-th is put into the upper
//      half of the k-th need, until all have one or no page is left;
//   3  the served needs go into the table, what they replace is given up;
//   4  the tokens' slots are read off the table.
// A sequence's count of needs is kept in lens_out until 4.
// 96 sequences of up to 9000 tokens in pages of 16, one new token each: 7.6 us, each step a
// round trip to memory.  Prompts, in pages of 16: one of 8191 tokens 9 us, 16 of 2048 29, one
// of 131072 68, of which step 4, 1024 slots at a time, is the most.
__global__ __launch_bounds__(kWide) void reserve_kernel(ReserveArgs a) {
    __shared__ int place[kWide + 1], entry[kWide], count[kWide];
    const int tid = threadIdx.x, mask = (1 << a.shift) - 1;
    const int64_t room = a.max_pages << a.shift;

    // the thread's sequence of the kWide from base on: where its tokens begin, how many, its length
    int floor = 0, start, n, len;
    bool fits;
    auto sequence = [&](int base) {
        const int b = base + tid;
        n = 0, len = 0;
        if (a.cu) {
            start = max(floor, group_scan_max<kWide>(b < a.B ? clamp_row(a.cu[b], a.total) : 0));
            if (b < a.B) n = max(clamp_row(a.cu[b + 1], a.total) - start, 0);
        } else {
            start = min(b, a.total);
            n = b < a.B ? 1 : 0;
        }
        if (b < a.B) len = (int)max((int64_t)0, min((int64_t)a.lens[b], room));
        fits = (int64_t)len + n <= room;
    };
    auto next_floor = [&]() {  // the last sequence's start bounds those of the next kWide
        __syncthreads();
        if (tid == kWide - 1) entry[0] = start;
        __syncthreads();
        floor = entry[0];
        __syncthreads();
    };

    // 1
    int needs = 0;
    for (int base = 0; base < a.B; base += kWide) {
        sequence(base);
        const int first = len >> a.shift, here = n > 0 && fits ? ((len + n + mask) >> a.shift) - first : 0;
        int all;
        const int before = group_scan<kWide>(here, &all);
        place[tid] = before, entry[tid] = first, count[tid] = 0;
        if (tid == 0) place[kWide] = all;
        __syncthreads();
        for (int k0 = 0; k0 < all; k0 += kWide) {
            const int k = k0 + tid;
            bool need = false;
            int i = 0;
            uint32_t at = 0;
            if (k < all) {
                // of equal places the last: the others have no entry
                i = last_at_most(place, kWide, k);
                at = (uint32_t)((int64_t)(base + i) * a.max_pages + entry[i] + k - place[i]);
                const uint32_t page = (uint32_t)a.table[at];
                need = page >= (uint64_t)a.pages || a.refs[page] > 1;
            }
            int found;
            const int rank = needs + group_scan<kWide>(need ? 1 : 0, &found);
            if (need) {
                a.slots[rank] = at;
                atomicAdd(&count[i], 1);
            }
            needs += found;
        }
        __syncthreads();
        if (base + tid < a.B) {
            a.lens_out[base + tid] = count[tid];
            *reinterpret_cast<int2 *>(a.copies + 2 * (int64_t)(base + tid)) = make_int2(-1, -1);
        }
        if (a.cu && a.B > kWide) next_floor();
        __syncthreads();
    }

    // 2
    constexpr int kPer = 16;  // pages of a thread at a time
    int given = 0;
    for (int64_t p0 = 0; p0 < a.pages && given < needs; p0 += kWide * kPer) {
        const int64_t p = p0 + tid * kPer;
        uint32_t unused = 0;
        if (p + kPer <= a.pages) {
            int4 r[kPer / 4];
#pragma unroll
            for (int i = 0; i < kPer / 4; ++i) r[i] = reinterpret_cast<const int4 *>(a.refs + p)[i];
#pragma unroll
            for (int i = 0; i < kPer / 4; ++i)
                unused |= (uint32_t)((r[i].x == 0) | (r[i].y == 0) << 1 | (r[i].z == 0) << 2 | (r[i].w == 0) << 3) << (4 * i);
        } else {
            for (int i = 0; i < kPer && p + i < a.pages; ++i) unused |= (uint32_t)(a.refs[p + i] == 0) << i;
        }
        int found;
        int rank = given + group_scan<kWide>(__popc(unused), &found);
        for (; unused != 0 && rank < needs; unused &= unused - 1, ++rank)
            reinterpret_cast<int32_t *>(a.slots + rank)[1] = (int32_t)(p + __builtin_ctz(unused));
        given = min(given + found, needs);
    }
    __syncthreads();

    // 3.  The needs are in order of the sequences: the first without a page names the
    // first sequence that is not served.
    auto entry_of = [&](int64_t need) { return (uint32_t)(uint64_t)need; };
    const int unserved = given < needs ? (int)(entry_of(a.slots[given]) / (uint32_t)a.max_pages) : a.B;
    for (int r = tid; r < given; r += kWide) {
        const int64_t need = a.slots[r];
        const uint32_t at = entry_of(need);
        const int b = (int)(at / (uint32_t)a.max_pages), page = (int)(need >> 32);
        if (b >= unserved) break;
        const int old = a.table[at];
        a.table[at] = page;
        a.refs[page] = 1;
        if ((uint32_t)old < (uint64_t)a.pages) {  // shared
            atomicSub(a.refs + old, 1);
            const int tokens = (int)max((int64_t)0, min((int64_t)a.lens[b], room));
            if ((tokens & mask) != 0 && (int64_t)b * a.max_pages + (tokens >> a.shift) == at)
                *reinterpret_cast<int2 *>(a.copies + 2 * (int64_t)b) = make_int2(old, page);
        }
    }
    __syncthreads();

    // 4
    floor = 0;
    int done = 0;
    for (int base = 0; base < a.B; base += kWide) {
        sequence(base);
        const int b = base + tid;
        bool served = false;
        if (b < a.B) {
            served = fits && (b < unserved || a.lens_out[b] == 0);
            a.lens_out[b] = served ? len + n : len;
        }
        place[tid] = start, entry[tid] = len, count[tid] = served ? n : 0;
        __syncthreads();
        const int last = min(kWide, a.B - base) - 1;
        // the tokens up to the last sequence's end; behind it those of the next kWide, or of nobody
        if (tid == last) place[kWide] = start + n;
        __syncthreads();
        const int end = base + kWide < a.B ? place[kWide] : a.total;
        for (int t = done + tid; t < end; t += kWide) {
            int64_t slot = -1;
            if (t >= place[0] && t < place[kWide]) {
                const int i = last_at_most(place, last + 1, t), pos = entry[i] + t - place[i];
                if (t - place[i] < count[i])
                    slot = ((int64_t)a.table[(int64_t)(base + i) * a.max_pages + (pos >> a.shift)] << a.shift) + (pos & mask);
            }
            a.slots[t] = slot;
        }
        done = max(done, end);
        if (a.cu && a.B > kWide) next_floor();
        __syncthreads();
    }
    for (int t = done + tid; t < a.total; t += kWide) a.slots[t] = -1;  // no sequences
}

// ------------------------------------------------------------------- fork --
constexpr int kForkColumns = 4096;  // of a workgroup

// The first B_out x chunks workgroups write the new rows and count their pages, the
// others give up the old rows' pages: additions to counts, whose order does not matter.
// 96 sequences of up to 9000 tokens in pages of 16: 5.9 us, the reads of a row's parent and
// its entries, then the counts.
__global__ __launch_bounds__(256) void fork_kernel(const int32_t *__restrict__ table, const int32_t *__restrict__ lens,
                                                   const int32_t *__restrict__ parents, int32_t *__restrict__ table_out,
                                                   int32_t *__restrict__ lens_out, int32_t *__restrict__ refs, int B,
                                                   int B_out, int64_t max_pages, int64_t pages, int shift, int chunks) {
    int row = (int)(blockIdx.x / (uint32_t)chunks);
    const int64_t first = (int64_t)(blockIdx.x - (uint32_t)row * chunks) * kForkColumns;
    const int64_t end = min(first + kForkColumns, max_pages);
    if (row >= B_out) {
        row -= B_out;
        for (int64_t c = first + threadIdx.x; c < end; c += 256) {
            const uint32_t page = (uint32_t)table[row * max_pages + c];
            if (page < (uint64_t)pages) atomicSub(refs + page, 1);
        }
        return;
    }
    const int parent = parents[row];
    int len = 0;
    if (parent >= 0 && parent < B) len = (int)max((int64_t)0, min((int64_t)lens[parent], max_pages << shift));
    const int64_t held = ((int64_t)len + (1 << shift) - 1) >> shift;
    if (first == 0 && threadIdx.x == 0) lens_out[row] = len;
    for (int64_t c = first + threadIdx.x; c < end; c += 256) {
        int page = -1;
        if (c < held) {
            page = table[parent * max_pages + c];
            if ((uint32_t)page < (uint64_t)pages)
                atomicAdd(refs + page, 1);
            else
                page = -1;
        }
        table_out[row * max_pages + c] = page;
    }
}

// ------------------------------------------------------------------- copy --
// A page's codes are one run of memory, its scales another.  A workgroup copies
// 16 KB of the codes (and the first also the scales), so that pages of any size
// spread over the card.  601 pages in 6 layers, 122 MB each way: 36 us on an input that
// the caches partly hold, 48 on a new one (5.0 TB/s).
constexpr int kCopyLoads = 4, kCopyBytes = 256 * 16 * kCopyLoads;

__global__ __launch_bounds__(256) void copy_kernel(uint8_t *__restrict__ codes, float *__restrict__ scales,
                                                   const int32_t *__restrict__ copies, int n, int chunks, int64_t pages,
                                                   int64_t page_bytes, int64_t page_scales) {
    const int pair = (int)(blockIdx.x / (uint32_t)chunks), chunk = (int)blockIdx.x - pair * chunks;
    const int layer = pair / n, i = pair - layer * n;
    const int2 c = *reinterpret_cast<const int2 *>(copies + 2 * (int64_t)i);
    if ((uint32_t)c.x >= (uint64_t)pages || (uint32_t)c.y >= (uint64_t)pages || c.x == c.y) return;
    const int64_t from = layer * pages + c.x, to = layer * pages + c.y;
    const uint4 *src = reinterpret_cast<const uint4 *>(codes + from * page_bytes);
    uint4 *dst = reinterpret_cast<uint4 *>(codes + to * page_bytes);
    const int64_t at = (int64_t)chunk * (kCopyBytes / 16) + threadIdx.x, end = page_bytes / 16;
    // the loads past the page's end read its last piece, so that none waits for a branch
    static_assert(kCopyLoads == 4);
    const uint4 w0 = src[min(at, end - 1)], w1 = src[min(at + 256, end - 1)], w2 = src[min(at + 512, end - 1)],
                w3 = src[min(at + 768, end - 1)];
    if (chunk == 0) {
        const float4 *s = reinterpret_cast<const float4 *>(scales + from * page_scales);
        float4 *d = reinterpret_cast<float4 *>(scales + to * page_scales);
        for (int64_t k = threadIdx.x; k < page_scales / 4; k += 256) d[k] = s[k];
    }
    if (at < end) dst[at] = w0;
    if (at + 256 < end) dst[at + 256] = w1;
    if (at + 512 < end) dst[at + 512] = w2;
    if (at + 768 < end) dst[at + 768] = w3;
}

// ---------------------------------------------------------------- compact --
struct CompactArgs {
    uint8_t *codes;
    float *scales;
    const int32_t *table, *lens, *cu;
    const uint8_t *keep;
    int32_t *lens_out;
    int B, total, H, shift;
    int64_t max_pages, pages;
    int64_t layer_rows;  // rows of one layer: pages 2 H page_size
    // many tokens, in the workspace: ...
    int4 *moves;  // ... for each its sequence, where it is, where it goes (-1: it stays), and the token there now
    int *ticket;  // ... how many units have been drawn
    int *read;    // ... whether a unit has read its rows, by the number of its launch
    // a launch: `layers` layers from layer0 on, the epoch-th, with `units` in each of those before
    int layer0, layers, epoch, units, groups, head_shift, token_shift;
};

// A sequence's new tokens: rows first .. first + n - 1 of `keep`, its cached length.
struct NewTokens {
    int first, n, len;
};
template <int kThreads>
__device__ __forceinline__ NewTokens new_tokens(const CompactArgs &a, int b) {
    NewTokens s = {b, 1, 0};
    if (a.cu) {
        __shared__ int top;
        int x = 0;  // the largest start up to its own
        for (int i = threadIdx.x; i <= b; i += kThreads) x = max(x, clamp_row(a.cu[i], a.total));
        x = group_scan_max<kThreads>(x);
        if (threadIdx.x == kThreads - 1) top = x;
        __syncthreads();
        s.first = top;
        s.n = max(clamp_row(a.cu[b + 1], a.total) - s.first, 0);
    }
    s.len = (int)max((int64_t)0, min((int64_t)a.lens[b], a.max_pages << a.shift));
    return s;
}

// The row of a token of sequence b, kv head h, keys or values, in one layer; -1: it has no page.
__device__ __forceinline__ int64_t row_of(const CompactArgs &a, const int32_t *table, int pos, int h, int which) {
    const uint32_t page = (uint32_t)table[pos >> a.shift];
    if (page >= (uint64_t)a.pages) return -1;
    return ((((int64_t)page * 2 + which) * a.H + h) << a.shift) + (pos & ((1 << a.shift) - 1));
}

// In place, by one workgroup for each sequence, head, keys or values and layer:
// 256 tokens at a time, whose kept rows are all read before the first is written.
// A kept token never moves up, so what is written has been read: it lies at or
// before the rows of its own 256 tokens, and those of later ones lie behind.
template <int D>
__global__ __launch_bounds__(256) void compact_kernel(CompactArgs a) {
    constexpr int kPieces = D / 16, kRows = 256 / kPieces;  // rows that the workgroup's threads take at once
    __shared__ int64_t from[256], to[256];
    const int tid = threadIdx.x;
    uint32_t item = blockIdx.x;
    const int which = item & 1;
    item >>= 1;
    const int h = (int)(item % (uint32_t)a.H);
    item /= (uint32_t)a.H;
    const int b = (int)(item % (uint32_t)a.B), layer = (int)(item / (uint32_t)a.B);
    const NewTokens s = new_tokens<256>(a, b);
    const int ctx = s.len - s.n;
    const int32_t *table = a.table + (int64_t)b * a.max_pages;
    uint4 *codes = reinterpret_cast<uint4 *>(a.codes + layer * a.layer_rows * D);
    float *scales = a.scales + layer * a.layer_rows;
    int dst = max(ctx, 0);
    for (int i0 = 0; i0 < s.n; i0 += 256) {
        const int i = i0 + tid, pos = ctx + i;
        const bool kept = i < s.n && pos >= 0 && a.keep[s.first + i] != 0;
        int all;
        const int rank = group_scan<256>(kept ? 1 : 0, &all);
        if (kept) {
            const int64_t src = row_of(a, table, pos, h, which);
            int64_t d = row_of(a, table, dst + rank, h, which);
            from[rank] = src, to[rank] = d == src ? -1 : d;
        }
        __syncthreads();
        uint4 w[256 / kRows];
        float scale = 0.0f;
#pragma unroll
        for (int k = 0; k < 256 / kRows; ++k) {
            const int r = tid / kPieces + kRows * k;
            w[k] = make_uint4(0, 0, 0, 0);
            if (r < all && to[r] >= 0 && from[r] >= 0) w[k] = codes[from[r] * kPieces + tid % kPieces];
        }
        if (tid < all && to[tid] >= 0 && from[tid] >= 0) scale = scales[from[tid]];
        // here before any wave writes
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 256 / kRows; ++k) {
            const int r = tid / kPieces + kRows * k;
            if (r < all && to[r] >= 0) codes[to[r] * kPieces + tid % kPieces] = w[k];
        }
        if (tid < all && to[tid] >= 0) scales[to[tid]] = scale;
        dst += all;
        __syncthreads();
    }
    if (layer == 0 && h == 0 && which == 0 && tid == 0) a.lens_out[b] = dst;
}

// For many tokens of few sequences, by all of the card: where each goes, and then their
// rows from one place to the other.  There are always starts: one token for each sequence
// is never more than compact_kernel takes.
constexpr int kChunkShift = 11, kChunkTokens = 1 << kChunkShift;

// The workgroup's sequence and 2048 of its new tokens: sequence b owns the workgroups
// from start / 2048 + b on, room for its tokens whatever their number.
struct Chunk {
    NewTokens s;
    int b, at, n;  // b < 0: nothing; tokens s.first + at .. + n - 1
};
__device__ __forceinline__ Chunk find_chunk(const CompactArgs &a) {
    const int lane = threadIdx.x & 63, rank = blockIdx.x;
    Chunk c = {{0, 0, 0}, -1, 0, 0};
    int first = 0, floor = 0;
    for (int base = 0; base < a.B; base += 64) {
        const int start = max(floor, wave_scan_max(base + lane < a.B ? clamp_row(a.cu[min(base + lane, a.B - 1)], a.total) : 0));
        const unsigned long long in = __ballot(base + lane < a.B && (start >> kChunkShift) + base + lane <= rank);
        if (in == 0) break;
        const int i = __popcll(in) - 1;
        c.b = base + i, first = __builtin_amdgcn_readlane(start, i);
        floor = __builtin_amdgcn_readlane(start, 63);
        if (in != ~0ull) break;
    }
    if (c.b < 0) return c;
    c.s.first = first, c.s.n = max(clamp_row(a.cu[c.b + 1], a.total) - first, 0);
    c.s.len = (int)max((int64_t)0, min((int64_t)a.lens[c.b], a.max_pages << a.shift));
    c.at = (rank - (first >> kChunkShift) - c.b) << kChunkShift;
    c.n = max(min(kChunkTokens, c.s.n - c.at), 0);
    if (c.at > 0 && c.n == 0) c.b = -1;  // every sequence has a first chunk, of no tokens perhaps
    return c;
}

// Whether token i of the chunk, which has some, stays; read whether or not there is a token i, so that a
// thread's loads are on their way together.
__device__ __forceinline__ bool stays(const CompactArgs &a, const Chunk &c, int i) {
    const uint8_t keep = a.keep[c.s.first + c.at + min(i, c.n - 1)];
    return (keep != 0) & (i < c.n) & (c.s.len - c.s.n + c.at + i >= 0);
}

// How many of n bytes are not zero, those that this thread of 256 takes: 16 at a time.
__device__ __forceinline__ int count_bytes(const uint8_t *p, int n) {
    const int head = min(n, (int)(-(uintptr_t)p & 15)), pieces = (n - head) / 16, tail = head + 16 * pieces;
    int sum = 0;
    if ((int)threadIdx.x < head) sum += p[threadIdx.x] != 0;
    if ((int)threadIdx.x < n - tail) sum += p[tail + threadIdx.x] != 0;
    const uint4 *words = reinterpret_cast<const uint4 *>(p + head);
    for (int i0 = threadIdx.x; i0 < pieces; i0 += 256 * 8) {
        uint4 w[8];  // on their way together
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = words[min(i0 + 256 * j, pieces - 1)];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t d[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
            int n16 = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) n16 += __popc((((d[k] & 0x7f7f7f7fu) + 0x7f7f7f7fu) | d[k]) & 0x80808080u);
            sum += i0 + 256 * j < pieces ? n16 : 0;
        }
    }
    return sum;
}

// Each workgroup counts the kept tokens before its own anew: with a launch that counts for all
// the call took 54 us for two contexts of 25,000 tokens in two layers, so 51 (this one 7 to 8), on an
// input that the caches partly hold.  The
// counting grows with the square of a sequence, for 2^20 tokens to some 3 % of the call.
__global__ __launch_bounds__(256) void compact_rank_kernel(CompactArgs a) {
    constexpr int kTurns = kChunkTokens / 256;
    __shared__ int waves[kTurns][4];
    __shared__ int top;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // the ticket and the flags of compact_move_kernel, which lie together, start from zeros
    for (int i = (int)blockIdx.x * 256 + tid; i <= a.units; i += (int)gridDim.x * 256) a.ticket[i] = 0;
    // rows of no sequence, by all workgroups: before the first start and from the largest on
    const int4 nowhere = make_int4(0, 0, -1, 0);
    int end = 0;
    for (int i = tid; i <= a.B; i += 256) end = max(end, clamp_row(a.cu[i], a.total));
    end = group_scan_max<256>(end);
    if (tid == 255) top = end;
    __syncthreads();
    const int first = clamp_row(a.cu[0], a.total), step = (int)gridDim.x * 256;
    for (int64_t t = blockIdx.x * 256 + tid; t < first; t += step) a.moves[t] = nowhere;
    for (int64_t t = (int64_t)top + blockIdx.x * 256 + tid; t < a.total; t += step) a.moves[t] = nowhere;
    const Chunk c = find_chunk(a);
    if (c.b < 0) return;
    bool kept[kTurns];
    int before[kTurns];
#pragma unroll
    for (int k = 0; k < kTurns; ++k) kept[k] = c.n > 0 && stays(a, c, 256 * k + tid);
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        const unsigned long long m = __ballot(kept[k]);
        before[k] = __popcll(m & ((1ull << lane) - 1));
        if (lane == 0) waves[k][wave] = __popcll(m);
    }
    // kept tokens of the sequence's chunks before this one, from its first that is there on
    const int ctx = c.s.len - c.s.n, there = min(max(-ctx, 0), c.at);
    int base;
    group_scan<256>(count_bytes(a.keep + c.s.first + there, c.at - there), &base);
    static_assert(kTurns * 4 <= 64, "one lane for each wave's turn");
    const int mine = lane < kTurns * 4 ? (&waves[0][0])[lane] : 0, upto = wave_scan(mine);
    const int all = __builtin_amdgcn_readlane(upto, 63), dst = max(ctx, 0) + base;
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        const int i = 256 * k + tid, from = ctx + c.at + i;
        const int to = dst + __shfl(upto - mine, 4 * k + wave, 64) + before[k];
        if (i < c.n) a.moves[c.s.first + c.at + i] = make_int4(c.b, from, kept[k] && to != from ? to : -1, c.s.first + to - ctx);
    }
    if (tid == 0 && c.at + c.n >= c.s.n) a.lens_out[c.b] = dst + all;
}

// In place, by many workgroups: a unit is 1024 rows (some tokens, the keys and values of
// up to 8 kv heads, one layer), read into registers and written where they go.  What is
// written over are rows of tokens before, so a unit first waits until the units that
// have those have read them.
// Each wait ends.  Units are given out in order of their tokens, by a ticket that a
// workgroup draws once it runs; a unit says that it has read before it waits for any
// other, and waits only for units of lower tickets: those run, and read without
// waiting.  Should calls overlap that share the workspace, which they must not, a wait
// ends after kPolls looks all the same (some 50 ms; a unit reads for a few us), and the
// sequence, whose rows are then lost, has the length -1.
// The rows of a token are read by its own unit alone, and other units write to them only
// after that, so no unit ever reads what another has written: a flag orders a read
// before a write, passes no data, and needs no cache written back.
// Half of 50,000 tokens of 8 heads of 128 channels in two layers, 211 MB: 59 us (3.6 TB/s) on an
// input that the caches do not hold, for each workgroup reads, then waits, then writes, and a
// CU has two.  On one that they partly hold 45, of which the waits are 4; in units of
// 256 rows 85, since all draw from one place (6 ns each); through memory in two steps 105.
constexpr int kUnitRows = 1024, kPolls = 1 << 16;

template <int D>
__global__ __launch_bounds__(1024) void compact_move_kernel(CompactArgs a) {
    constexpr int kPieces = D / 16, kRows = 1024 / kPieces, kPasses = kUnitRows / kRows;
    __shared__ int64_t from[kUnitRows / 2], to[kUnitRows / 2];  // of keys of head 0; from -1: zeros; to -1: nothing to do
    __shared__ int drawn;
    const int tid = threadIdx.x, piece = tid % kPieces, heads = 1 << a.head_shift, lanes = a.layers * a.groups;
    if (tid == 0) drawn = (int)((uint32_t)atomicAdd(a.ticket, 1) - (uint32_t)a.epoch * (uint32_t)a.units);
    __syncthreads();
    const int unit = drawn;
    if ((uint32_t)unit >= gridDim.x) return;  // calls that overlap, as below
    // the unit's tokens: `chunk` of 2^token_shift; its kv heads: `group` of 2^head_shift
    const int chunk = unit / lanes, lane = unit - chunk * lanes;
    const int layer = lane / a.groups, group = lane - layer * a.groups;
    const int t0 = chunk << a.token_shift, n = min(1 << a.token_shift, a.total - t0);
    int over = -1;  // the chunk whose row this thread's token is written over
    if (tid < n) {
        const int4 move = a.moves[t0 + tid];
        // always so where it moves, but for calls that overlap: those spoil each other's rows, and reach no others
        const uint32_t room = (uint32_t)(a.max_pages << a.shift);
        const bool moves = move.z >= 0 && (uint32_t)move.z < room && (uint32_t)move.y < room && (uint32_t)move.x < (uint32_t)a.B;
        const int32_t *table = a.table + (moves ? move.x * a.max_pages : 0);
        from[tid] = moves ? row_of(a, table, move.y, 0, 0) : -1;
        to[tid] = moves ? row_of(a, table, move.z, 0, 0) : -1;
        if (moves) over = move.w >> a.token_shift;
    }
    __syncthreads();
    uint4 *codes = reinterpret_cast<uint4 *>(a.codes + (a.layer0 + layer) * a.layer_rows * D);
    float *scales = a.scales + (a.layer0 + layer) * a.layer_rows;
    // row r of the unit: token r >> (head_shift + 1), then keys and values, then heads
    int64_t dst[kPasses];
    uint4 w[kPasses];
    float scale[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int r = kRows * p + tid / kPieces, token = r >> (a.head_shift + 1), kind = r & (2 * heads - 1);
        const int h = (group << a.head_shift) + (kind & (heads - 1));
        const int64_t at = (int64_t)((kind >> a.head_shift) * a.H + h) << a.shift;
        const bool mine = token < n && h < a.H && to[min(token, n - 1)] >= 0;
        const int64_t src = mine ? from[token] : -1;
        dst[p] = mine ? to[token] + at : -1;
        w[p] = src >= 0 ? codes[(src + at) * kPieces + piece] : make_uint4(0, 0, 0, 0);
        scale[p] = src >= 0 && piece == 0 ? scales[src + at] : 0.0f;
    }
    // read: the loads have come back before the unit says so; the compiler sees them arrive
    // here too, or it would wait for each store before the next
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
    for (int p = 0; p < kPasses; ++p) asm volatile("" : "+v"(w[p].x), "+v"(w[p].y), "+v"(w[p].z), "+v"(w[p].w), "+v"(scale[p]));
    __syncthreads();
    if (tid == 0) __hip_atomic_store(a.read + unit, a.epoch + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (over >= 0 && over < chunk) {
        const int *other = a.read + over * lanes + lane;
        auto seen = [&]() { return __hip_atomic_load(other, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) > a.epoch; };
        if (!wait_until(seen, []() { __builtin_amdgcn_s_sleep(1); }, kPolls)) {
            const int b = a.moves[t0 + tid].x;  // anew, as a register for it would leave a CU room for one workgroup, not two
            if ((uint32_t)b < (uint32_t)a.B) a.lens_out[b] = -1;
        }
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        if (dst[p] < 0) continue;
        codes[dst[p] * kPieces + piece] = w[p];
        if (piece == 0) scales[dst[p]] = scale[p];
    }
}

constexpr int64_t kMostUnits = int64_t(1) << 21;  // of a launch of 1024 threads each

template <int D>
qw3_status launch_compact(CompactArgs a, int64_t layers, hipStream_t stream) {
    const int64_t items = layers * a.B * a.H * 2;
    // One workgroup per head takes 256 tokens at a time, one after the other.  The host knows the
    // average alone: 20,000 tokens of one sequence are moved in 40 us, among 63 sequences without
    // any in 223.
    if (a.total <= 512 * (int64_t)a.B) {
        if (items >= kMaxGroups) return QW3_ERR_SHAPE;
        hipLaunchKernelGGL((compact_kernel<D>), dim3((unsigned)items), dim3(256), 0, stream, a);
        return check_launch();
    }
    // heads of a unit: up to 8, a power of two; its tokens: as many as make 1024 rows
    while (a.head_shift < 3 && (1 << a.head_shift) < a.H) ++a.head_shift;
    a.token_shift = 9 - a.head_shift;
    a.groups = (int)ceil_div(a.H, 1 << a.head_shift);
    const int64_t chunks = ceil_div(a.total, 1 << a.token_shift);
    if (a.total * ((int64_t)a.groups << a.head_shift) >= int64_t(1) << 30) return QW3_ERR_SHAPE;  // 2^21 + 128 units a layer
    int64_t some = kMostUnits / (chunks * a.groups);  // layers at a time
    some = some < 1 ? 1 : some < layers ? some : layers;
    const int64_t units = chunks * a.groups * some;
    a.units = (int)units;
    const int64_t ranks = (a.total >> kChunkShift) + a.B;
    Scratch ws;
    const qw3_status st = workspace(stream, (size_t)(a.total * int64_t(16) + (1 + units) * int64_t(4)), &ws);
    if (st != QW3_OK) return st;
    a.moves = static_cast<int4 *>(ws.ptr);
    a.ticket = reinterpret_cast<int *>(a.moves + a.total), a.read = a.ticket + 1;
    hipLaunchKernelGGL(compact_rank_kernel, dim3((unsigned)ranks), dim3(256), 0, stream, a);
    for (; a.layer0 < layers; a.layer0 += (int)some, ++a.epoch) {
        a.layers = (int)(some < layers - a.layer0 ? some : layers - a.layer0);
        hipLaunchKernelGGL((compact_move_kernel<D>), dim3((unsigned)(chunks * a.groups * a.layers)), dim3(1024), 0, stream, a);
    }
    return check_launch();
}

// What the calls on block tables check; *shift = log2(page_size).
qw3_status check_tables(int64_t B, int64_t max_pages, int64_t pages, int64_t page_size, int *shift) {
    const qw3_status st = check_cache(QW3_CODES_INT8, 1, 64, pages, page_size, shift);
    if (st != QW3_OK) return st;
    if (B < 0 || B > QW3_MAX_SEQS || max_pages < 0 || max_pages > (int64_t(1) << 30) / page_size) return QW3_ERR_SHAPE;
    return B * max_pages < (int64_t(1) << 32) ? QW3_OK : QW3_ERR_SHAPE;
}

}  // namespace

extern "C" {

qw3_status qcache_reserve(int32_t *refs, int32_t *block_table, const int32_t *lens, const int32_t *cu, int64_t *slots,
                          int32_t *lens_out, int32_t *copies, int64_t B, int64_t max_pages, int64_t total,
                          int64_t pages, int64_t page_size, void *hip_stream) {
    int shift = 0;
    const qw3_status st = check_tables(B, max_pages, pages, page_size, &shift);
    if (st != QW3_OK) return st;
    if (total < 0 || total > QW3_MAX_TOKENS || (!cu && total != B)) return QW3_ERR_SHAPE;
    if (B == 0 && total == 0) return QW3_OK;
    if ((B > 0 && (!lens || !lens_out || !copies)) || (B > 0 && max_pages > 0 && !block_table) || (pages > 0 && !refs) ||
        (total > 0 && !slots))
        return QW3_ERR_NULL;
    if (!aligned(refs, 16) || !aligned(block_table, 4) || !aligned(lens, 4) || !aligned(cu, 4) || !aligned(slots, 8) ||
        !aligned(lens_out, 4) || !aligned(copies, 8))
        return QW3_ERR_ALIGN;
    ReserveArgs a{};
    a.refs = refs, a.table = block_table, a.lens = lens, a.cu = cu, a.slots = slots, a.lens_out = lens_out;
    a.copies = copies, a.B = (int)B, a.total = (int)total, a.shift = shift, a.max_pages = max_pages, a.pages = pages;
    hipLaunchKernelGGL(reserve_kernel, dim3(1), dim3(kWide), 0, (hipStream_t)hip_stream, a);
    return check_launch();
}

qw3_status qcache_fork(int32_t *refs, const int32_t *block_table, const int32_t *lens, const int32_t *parents,
                       int32_t *table_out, int32_t *lens_out, int64_t B, int64_t B_out, int64_t max_pages, int64_t pages,
                       int64_t page_size, void *hip_stream) {
    int shift = 0;
    qw3_status st = check_tables(B, max_pages, pages, page_size, &shift);
    if (st != QW3_OK) return st;
    st = check_tables(B_out, max_pages, pages, page_size, &shift);
    if (st != QW3_OK) return st;
    // at most 2^17 rows and 2^32 entries of each table: the grid stays below 2^22 workgroups
    const int64_t chunks = max_pages > kForkColumns ? ceil_div(max_pages, kForkColumns) : 1;
    if (B + B_out == 0) return QW3_OK;
    if ((B > 0 && !lens) || (B > 0 && max_pages > 0 && !block_table) || (B_out > 0 && (!parents || !lens_out)) ||
        (B_out > 0 && max_pages > 0 && !table_out) || (pages > 0 && !refs))
        return QW3_ERR_NULL;
    if (!aligned(refs, 16) || !aligned(block_table, 4) || !aligned(lens, 4) || !aligned(parents, 4) ||
        !aligned(table_out, 4) || !aligned(lens_out, 4))
        return QW3_ERR_ALIGN;
    hipLaunchKernelGGL(fork_kernel, dim3((unsigned)((B + B_out) * chunks)), dim3(256), 0, (hipStream_t)hip_stream,
                       block_table, lens, parents, table_out, lens_out, refs, (int)B, (int)B_out, max_pages, pages, shift,
                       (int)chunks);
    return check_launch();
}

qw3_status qcache_copy(void *codes, float *scales, const int32_t *copies, int64_t n, int64_t layers, int64_t H, int64_t D,
                       int64_t pages, int64_t page_size, void *hip_stream) {
    int shift = 0;
    const qw3_status st = check_cache(QW3_CODES_INT8, H, D, pages, page_size, &shift);
    if (st != QW3_OK) return st;
    if (n < 0 || n > QW3_MAX_TOKENS || layers < 0 || layers > QW3_MAX_LAYERS) return QW3_ERR_SHAPE;
    const int64_t bytes = 2 * H * D << shift, chunks = ceil_div(bytes, kCopyBytes);
    if (n * layers * chunks >= kMaxGroups) return QW3_ERR_SHAPE;
    if (n == 0 || layers == 0 || pages == 0) return QW3_OK;
    if (!codes || !scales || !copies) return QW3_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(copies, 8)) return QW3_ERR_ALIGN;
    hipLaunchKernelGGL(copy_kernel, dim3((unsigned)(n * layers * chunks)), dim3(256), 0, (hipStream_t)hip_stream,
                       static_cast<uint8_t *>(codes), scales, copies, (int)n, (int)chunks, pages, bytes, 2 * H << shift);
    return check_launch();
}

qw3_status qcache_compact(void *codes, float *scales, const int32_t *block_table, const int32_t *lens, const int32_t *cu_q,
                          const uint8_t *keep, int32_t *lens_out, int64_t B, int64_t max_pages, int64_t Tq,
                          int64_t layers, int64_t H, int64_t D, int64_t pages, int64_t page_size, void *hip_stream) {
    int shift = 0;
    qw3_status st = check_cache(QW3_CODES_INT8, H, D, pages, page_size, &shift);
    if (st != QW3_OK) return st;
    st = check_tables(B, max_pages, pages, page_size, &shift);
    if (st != QW3_OK) return st;
    if (Tq < 0 || Tq > QW3_MAX_TOKENS || (!cu_q && Tq != B) || layers < 1 || layers > QW3_MAX_LAYERS) return QW3_ERR_SHAPE;
    if (layers * B * H * 2 >= kMaxGroups) return QW3_ERR_SHAPE;
    if (B == 0) return QW3_OK;
    if (!lens || !lens_out || (Tq > 0 && !keep) || (max_pages > 0 && !block_table) || (pages > 0 && (!codes || !scales)))
        return QW3_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(block_table, 4) || !aligned(lens, 4) || !aligned(cu_q, 4) ||
        !aligned(lens_out, 4))
        return QW3_ERR_ALIGN;
    CompactArgs a{};
    a.codes = static_cast<uint8_t *>(codes), a.scales = scales, a.table = block_table, a.lens = lens, a.cu = cu_q;
    a.keep = keep, a.lens_out = lens_out, a.B = (int)B, a.total = (int)Tq, a.H = (int)H, a.shift = shift;
    a.max_pages = max_pages, a.pages = pages, a.layer_rows = pages * 2 * H << shift;
    return D == 128 ? launch_compact<128>(a, layers, (hipStream_t)hip_stream)
                    : launch_compact<64>(a, layers, (hipStream_t)hip_stream);
}

}  // extern "C"
