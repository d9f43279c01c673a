// Attention over some of the cache's pages: the bounds of each page's keys
// (qcache_bounds), the pages that a cheap score by them selects for each query and
// kv head (qblock_select), and attention over those (qattn_blocks).  C ABI in
// include/qw3.h.
//
// Bounds.  Per page and kv head, channel d of the keys' values x = c s (fp32) lies
// between mn_d and mx_d; both are kept as int8 under one scale S = max |.| / 127.
// Score.  With u_d = sum over the head's queries of max(q_d, 0) and n_d of min(q_d,
// 0), sum_d u_d mx_d + n_d mn_d is at least the sum of their scores of any key of
// the page.  u and n are kept as int8 under one scale too, which does not change
// the order of the pages; so a score is a whole number below 2^24 times S, one
// rounding, the same in whatever order it is summed: the selection is a matter of
// definition, not of the kernel.
#include "qw3_attn_dev.h"

using namespace qw3_shared;

namespace {

// The sequence, the place in it and the position of a packed row: the row is token
// len - n + i.  A wave's lanes together; b < 0: a row of no sequence.
struct Row {
    int b, pos, len;
};
__device__ __forceinline__ Row find_row(const int32_t *cu, const int32_t *lens, int B, int total, int64_t room, int t) {
    const int lane = threadIdx.x & 63;
    auto length = [&](int b) { return (int)max((int64_t)0, min((int64_t)lens[b], room)); };
    if (cu == nullptr) {
        const int len = length(t);
        return Row{t, len - 1, len};
    }
    Row row = {-1, 0, 0};
    int floor = 0;
    for (int base = 0; base < B; base += 64) {
        const int start = max(floor, wave_scan_max(base + lane < B ? clamp_row(cu[min(base + lane, B - 1)], total) : 0));
        const unsigned long long in = __ballot(base + lane < B && start <= t);
        if (in == 0) break;
        const int at = __popcll(in) - 1;  // the starts do not fall, so these are the first lanes
        row.b = base + at, row.pos = __builtin_amdgcn_readlane(start, at);
        floor = __builtin_amdgcn_readlane(start, 63);
        if (in != ~0ull) break;
    }
    row.b = uniform(row.b);
    if (row.b < 0) return row;
    const int first = uniform(row.pos), end = clamp_row(cu[row.b + 1], total);
    row.len = length(row.b);
    row.pos = row.len - (end - first) + t - first;
    if (t >= end) row.b = -1;
    return row;
}

// ----------------------------------------------------------------- bounds --
struct BoundsArgs {
    const uint8_t *codes;
    const float *scales;
    const int32_t *table, *lens, *cu;
    int8_t *bounds;
    float *steps;
    int B, Tq, H, shift, items;
    int64_t max_pages, pages;
};

// The larger of two numbers that come as bits from other lanes: the middle one of them and
// +inf, since of a maximum the compiler would first make quiet NaN of each, which costs as
// much again; a NaN that is lost here has been seen before.  Not in asm: what an exchange
// between lanes reads has to be two instructions old, which the compiler sees to for its own.
struct Larger {
    float inf = __builtin_huge_valf();
    __device__ __forceinline__ Larger() { asm("" : "+s"(inf)); }  // a constant would make it a maximum again
    __device__ __forceinline__ float operator()(uint32_t x, uint32_t y) const {
        return __builtin_amdgcn_fmed3f(__uint_as_float(x), __uint_as_float(y), inf);
    }
    // of what lanes l and l ^ 8 (l ^ 4) of each 16 hold, in both
    __device__ __forceinline__ float ror8(float x) const { return (*this)(__float_as_uint(x), __float_as_uint(dpp_f32<0x128>(x))); }
    __device__ __forceinline__ float ror4(float x) const { return (*this)(__float_as_uint(x), __float_as_uint(dpp_f32<0x124>(x))); }
};

// A wave has one page and head.  D / 16 lanes take a row, 16 channels each, and the
// wave 1024 / D rows at a time; what lanes of the same channels hold is joined at the
// end, halving in each step the channels that a lane stands for.  30,001 tokens of 8 heads
// of 128 channels in pages of 32, e4m3: 9.9 us (11 on an input that the caches do not hold), 33
// MB at 3.3 TB/s; vector instructions are issued 64 % of the time.  A page's 32 rows take a wave
// some 480 of them, 7.5 for each of a lane's 64 codes: conversions, products and maxima are 160, the
// NaN test of e4m3 codes 40, the joins across lanes 130, quotients and codes 75, finding the
// sequence 40, addresses the rest.
template <int D, bool E4M3>
__global__ __launch_bounds__(256) void bounds_kernel(BoundsArgs a) {
    constexpr int kPieces = D / 16, kRows = 64 / kPieces;
    const int lane = threadIdx.x & 63;
    const int unit = (int)blockIdx.x * 4 + uniform((int)threadIdx.x >> 6);
    const int item = (int)((uint32_t)unit / (uint32_t)a.H), h = unit - item * a.H;
    if (item >= a.items) return;
    // Sequence b owns the items from start / page_size + 2 b on: room for its pages whatever its length.
    const int64_t room = a.max_pages << a.shift;
    int b = item, n = 1, at = 0, len = 0;
    if (a.cu != nullptr) {
        int first = 0, end = 0, floor = 0;
        b = -1;
        for (int base = 0; base < a.B; base += 64) {
            // what a lane's sequence would need, read at once
            const int mine = min(base + lane, a.B - 1), until = clamp_row(a.cu[mine + 1], a.Tq), length = a.lens[mine];
            const int start = max(floor, wave_scan_max(base + lane < a.B ? clamp_row(a.cu[mine], a.Tq) : 0));
            const unsigned long long in = __ballot(base + lane < a.B && (start >> a.shift) + 2 * (base + lane) <= item);
            if (in == 0) break;
            const int i = __popcll(in) - 1;
            b = base + i, first = __builtin_amdgcn_readlane(start, i), end = __builtin_amdgcn_readlane(until, i);
            len = __builtin_amdgcn_readlane(length, i);
            floor = __builtin_amdgcn_readlane(start, 63);
            if (in != ~0ull) break;
        }
        b = uniform(b), first = uniform(first);
        if (b < 0) return;
        n = uniform(end) - first;
        at = item - (first >> a.shift) - 2 * b;
    } else {
        len = a.lens[b];
    }
    if (n <= 0) return;
    len = uniform((int)max((int64_t)0, min((int64_t)len, room)));
    const int64_t col = (max(len - n, 0) >> a.shift) + (int64_t)at;
    if (col << a.shift >= len) return;
    const uint32_t page = (uint32_t)uniform(a.table[b * a.max_pages + col]);
    if (page >= (uint64_t)a.pages) return;
    const int count = min(1 << a.shift, len - (int)(col << a.shift));

    const int piece = lane % kPieces;
    const int64_t row0 = ((int64_t)page * 2 * a.H + h) << a.shift;
    const uint8_t *codes = a.codes + row0 * D + piece * 16;
    const float *scales = a.scales + row0;
    float v[32];  // the channels' largest values, then those of the values' opposites
    uint32_t nans = 0;
    float worst = 0.0f;
    constexpr int kAt = 32 / kRows;  // 32 rows on their way together, compared in twos
    auto rows32 = [&](int base, auto first_c) {
        uint4 w[kAt];
        float s[kAt];
#pragma unroll
        for (int k = 0; k < kAt; ++k) {
            const int r = min(base + k * kRows + lane / kPieces, count - 1);  // the last row again does no harm
            w[k] = *reinterpret_cast<const uint4 *>(codes + (int64_t)r * D);
            s[k] = scales[r];
        }
#pragma unroll
        for (int k = 0; k < kAt; k += 2) {
            constexpr bool kFirst = decltype(first_c)::value;
            if (k > 0 && base + k * kRows >= count) break;
            const uint32_t d[2][4] = {{w[k].x, w[k].y, w[k].z, w[k].w}, {w[k + 1].x, w[k + 1].y, w[k + 1].z, w[k + 1].w}};
            worst += s[k] * 0.0f + s[k + 1] * 0.0f;  // stays 0 unless a scale is not finite
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float f[2][4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (E4M3) {
                        nans |= (d[j][i] & 0x7f7f7f7fu) + 0x01010101u;
                        const f2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(d[j][i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(d[j][i], true);
                        f[j][0] = lo[0], f[j][1] = lo[1], f[j][2] = hi[0], f[j][3] = hi[1];
                    } else {
                        f[j][0] = byte_f32<0>(d[j][i]), f[j][1] = byte_f32<1>(d[j][i]);
                        f[j][2] = byte_f32<2>(d[j][i]), f[j][3] = byte_f32<3>(d[j][i]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = f[0][e] * s[k], y = f[1][e] * s[k + 1];
                    v[4 * i + e] = kFirst && k == 0 ? fmaxf(x, y) : fmaxf(fmaxf(x, y), v[4 * i + e]);
                    v[16 + 4 * i + e] = kFirst && k == 0 ? fmaxf(-x, -y) : fmaxf(fmaxf(-x, -y), v[16 + 4 * i + e]);
                }
            }
        }
    };
    rows32(0, std::true_type{});
    for (int base = 32; base < count; base += 32) rows32(base, std::false_type{});
    const bool bad = !(worst == 0.0f);
    const Larger larger;
    // lanes 0..31 keep the maxima, the others those of the opposites; then the even
    // sixteens of lanes the first 8 channels, the odd ones the last
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[16 + i]), false, false);
        v[i] = larger(r[0], r[1]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]), __float_as_uint(v[8 + i]), false, false);
        v[i] = larger.ror8(larger(r[0], r[1]));
        if (D == 64) v[i] = larger.ror4(v[i]);
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    top = (uint32_t)wave_max((int)top);
    const bool finite = top < 0x7f800000u && !__any(bad || (nans & 0x80808080u) != 0);
    const float step = finite ? __uint_as_float(top) / 127.0f : __uint_as_float(0x7fc00000u);
    // quotients as in qw3_quant.h; the sign of those of the opposites goes into the divisor
    float y[8];
    const float divisor = lane < 32 ? step : -step;
    if (step > 0x1p-80f && step < 0x1p100f) {
        const float r = 1.0f / divisor;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float q = v[i] * r;
            q = fmaf(fmaf(-q, divisor, v[i]), r, q);
            y[i] = fmaf(fmaf(-q, divisor, v[i]), r, q);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = step > 0.0f ? fminf(fmaxf(v[i] / divisor, -127.0f), 127.0f) : 0.0f;
    }
    const uint32_t lo = codes4<false>({y[0], y[1], y[2], y[3]}), hi = codes4<false>({y[4], y[5], y[6], y[7]});
    const int64_t to = (int64_t)page * a.H + h;
    if ((lane & 15) < kPieces)
        *reinterpret_cast<uint2 *>(a.bounds + (to * 2 + (lane >> 5)) * D + 16 * piece + 8 * ((lane >> 4) & 1)) = make_uint2(lo, hi);
    if (lane == 0) a.steps[to] = step;
}

// ----------------------------------------------------------------- select --
struct SelectArgs {
    const uint16_t *q;
    const int8_t *bounds;
    const float *steps;
    const int32_t *table, *lens, *cu;
    int32_t *picks;
    uint32_t *keys;  // in memory: those of the launch's rows, [rows, H, pitch]
    int *counts, *clear;  // how many workgroups of a row and kv head have finished, and the next call's counters
    int64_t q_ts, q_hs, max_pages, pages;
    int B, Tq, H, G, shift, count, first, recent, pitch;
    int t0, rows;  // the rows of a launch: from t0 on
};

// A score as a number that orders like it; NaN above all, 0 for a page that is not there.
__device__ __forceinline__ uint32_t key_of(float score) {
    const uint32_t u = __float_as_uint(score + 0.0f);  // no negative zero
    if ((u & 0x7fffffffu) > 0x7f800000u) return ~0u;
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
constexpr uint32_t kNoPage = ~0u;  // in the place of a page's step

// The w of row `row` for kv head h as int8 [2 D] in LDS, by one wave, D / 64 channels
// of every query a lane.
template <int D>
__device__ __forceinline__ void query_codes(const SelectArgs &a, int row, int h, uint8_t *w) {
    constexpr int kPer = D / 64;
    const int lane = threadIdx.x & 63;
    double u[kPer] = {}, l[kPer] = {};
    const uint16_t *q = a.q + (int64_t)row * a.q_ts + (int64_t)h * a.G * a.q_hs + kPer * lane;
    // in 64 bits and in the queries' order, which is part of the definition: what lies more than
    // 53 bits below another is rounded away
#pragma unroll 8
    for (int g = 0; g < a.G; ++g) {
        const uint32_t d = kPer == 2 ? *reinterpret_cast<const uint32_t *>(q + g * a.q_hs) : (uint32_t)q[g * a.q_hs] << 16;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const float f = __uint_as_float(kPer == 2 && i == 0 ? d << 16 : d & 0xffff0000u);
            // a NaN into both sums
            u[i] += f < 0.0f ? 0.0 : (double)f;
            l[i] += f > 0.0f ? 0.0 : (double)f;
        }
    }
    float x[2][kPer];
    auto round_all = [&](double times) {  // the largest, as bits
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            x[0][i] = (float)(u[i] * times), x[1][i] = (float)(l[i] * times);
            top = max(top, max(__float_as_uint(x[0][i]) & 0x7fffffffu, __float_as_uint(x[1][i]) & 0x7fffffffu));
        }
        return (uint32_t)wave_max((int)top);
    };
    uint32_t top = round_all(1.0);
    // finite queries may add up to more than fp32 holds; the scale of u and n is nobody's
    static_assert(QW3_MAX_HEADS <= 1 << 15, "2^128 each");
    if (top >= 0x7f800000u) top = round_all(0x1p-16);
    const float s = top < 0x7f800000u ? __uint_as_float(top) / 127.0f : 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float y[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kPer; ++i) y[i] = s > 0.0f ? fminf(fmaxf(x[k][i] / s, -127.0f), 127.0f) : 0.0f;
        const uint32_t c = codes4<false>({y[0], y[1], 0.0f, 0.0f});
        if (kPer == 2)
            *reinterpret_cast<uint16_t *>(w + k * D + 2 * lane) = (uint16_t)c;
        else
            w[k * D + lane] = (uint8_t)c;
    }
}

// The page numbers of a wave's 64 pages from p on, one for each lane.
__device__ __forceinline__ uint32_t page_at(const SelectArgs &a, const int32_t *table, int p) {
    return a.max_pages == 0 ? kNoPage : (uint32_t)table[min((int64_t)p + (threadIdx.x & 63), a.max_pages - 1)];
}

// Keys of the pages from p on below `pages`, 64 for each step of `stride` pages, by one wave;
// page: page_at(p).  The matrix unit's rows are 16 pages, its columns the kRows rows' w,
// which prepare() sees to, once the first pages are on their way.
// put(row, page, keys): the keys of 4 pages from one on, for the first n rows.
template <int D, int kRows, class Prepare, class Put>
__device__ __forceinline__ void score_pages(const SelectArgs &a, const int32_t *table, int h, int p, int stride, int pages, int n,
                                            uint32_t page, const uint8_t *w, Prepare prepare, Put put) {
    constexpr int kSteps = 2 * D / 64;
    const int lane = threadIdx.x & 63, col = lane & 15, quarter = lane >> 4;
    uint32_t step;
    i4_t kf[4][kSteps];
    auto load = [&]() {  // one page's step a lane, then the bounds of 64 pages on their way together
        step = kNoPage;
        if (page < (uint64_t)a.pages) {
            step = __float_as_uint(a.steps[(int64_t)page * a.H + h]);
            if (step == kNoPage) step = 0x7fc00000u;
        } else {
            page = kNoPage;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t id = (uint32_t)__shfl((int)page, 16 * j + col, 64);
#pragma unroll
            for (int k = 0; k < kSteps; ++k) kf[j][k] = i4_t{};
            if (id != kNoPage && p + 16 * j < pages) {
                const int8_t *at = a.bounds + ((int64_t)id * a.H + h) * 2 * D + 16 * quarter;
#pragma unroll
                for (int k = 0; k < kSteps; ++k) kf[j][k] = *reinterpret_cast<const i4_t *>(at + 64 * k);
            }
        }
    };
    if (p < pages) load();
    prepare();
    i4_t wf[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
        wf[k] = *reinterpret_cast<const i4_t *>(w + (kRows == 1 ? 0 : col) * 2 * D + 64 * k + 16 * quarter);
    while (p < pages) {
        const int at = p;
        p += stride;
        if (p < pages) page = page_at(a, table, p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            i4_t sum = {};
#pragma unroll
            for (int k = 0; k < kSteps; ++k) sum = __builtin_amdgcn_mfma_i32_16x16x64_i8(kf[j][k], wf[k], sum, 0, 0, 0);
            uint32_t key[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t s = (uint32_t)__shfl((int)step, 16 * j + 4 * quarter + r, 64);
                key[r] = s == kNoPage ? 0u : key_of((float)sum[r] * __uint_as_float(s));
            }
            if (col < n && at + 16 * j < pages)
                put(col, at + 16 * j + 4 * quarter, make_uint4(key[0], key[1], key[2], key[3]));
        }
        if (p < pages) load();
    }
}

template <int T>
__device__ __forceinline__ void group_sync() {
    if constexpr (T > 64) {
        __syncthreads();
    } else {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// What T threads need to pick: a histogram of 256 for each byte, and what waves exchange.
// bins are cleared and summed 16 bytes at a time, in each PickSpace of an array.
template <int T>
struct alignas(16) PickSpace {
    int bins[T > 64 ? 4 : 1][256];
    uint32_t waves[2][T / 64];
    int taken[T > 64 ? 64 : 1];
};

// A row's picks out of `seen` pages, by T threads whose number among them is tid.
// All if there are at most count; else the first ones, the last ones, and of those
// between the `left` with the largest keys.  The left-th largest key is found by 8 bits at
// a time, below the bits that all keys have in common, in counts of the keys that have the
// bits found so far; then the pages are gone through in order, and of those with that key
// the first are taken.
// key_at(i): page i's key; up to kHeld T of them are kept, more are read anew in each pass.
template <int T, int kHeld, class Key>
__device__ __forceinline__ void pick(const SelectArgs &a, Key key_at, int seen, int32_t *out, PickSpace<T> &space, int tid) {
    if (seen <= a.count) {
        for (int i = tid; i < a.count; i += T) out[i] = i < seen ? i : -1;
        return;
    }
    const int lane = tid & 63, wave = tid >> 6, lo = a.first, hi = seen - a.recent;
    int left = a.count - a.first - a.recent;
    const bool none = left <= 0;
    constexpr int kWaves = T / 64;
    const bool held = hi - lo <= kHeld * T;
    uint32_t kept[kHeld];
#pragma unroll
    for (int j = 0; j < kHeld; ++j) kept[j] = key_at(min(lo + tid + T * j, hi - 1));
    auto each = [&](auto f) {
        if (held) {
#pragma unroll
            for (int j = 0; j < kHeld; ++j)
                if (lo + tid + T * j < hi) f(kept[j]);
        } else {
            for (int i = lo + tid; i < hi; i += T) f(key_at(i));
        }
    };
    uint32_t prefix = 0, mask = 0;
    if (!none) {
        uint32_t all = ~0u, any = 0;
        each([&](uint32_t key) { all &= key, any |= key; });
#pragma unroll
        for (int m = 32; m >= 1; m /= 2) all &= (uint32_t)__shfl_xor((int)all, m, 64), any |= (uint32_t)__shfl_xor((int)any, m, 64);
        if constexpr (T > 64) {
            if (lane == 0) space.waves[0][wave] = all, space.waves[1][wave] = any;
            for (int i = tid; i < 4 * 256; i += T) space.bins[0][i] = 0;
            __syncthreads();
#pragma unroll
            for (int x = 0; x < T / 64; ++x) all &= space.waves[0][x], any |= space.waves[1][x];
        }
        int shift = 32 - (all == any ? 32 : __builtin_clz(all ^ any));  // of the lowest bit found so far
        mask = shift == 32 ? 0u : ~0u << shift, prefix = all & mask;
        for (int pass = 0; shift > 0; ++pass) {
            const int width = min(shift, 8);
            shift -= width;
            int *bins = space.bins[T > 64 ? pass : 0];
            if constexpr (T == 64) {
                group_sync<T>();
                *reinterpret_cast<int4 *>(bins + 4 * lane) = make_int4(0, 0, 0, 0);
                group_sync<T>();
            }
            each([&](uint32_t key) {
                if ((key & mask) == prefix) atomicAdd(bins + (key >> shift & ((1u << width) - 1)), 1);
            });
            group_sync<T>();
            // by every wave: lane l has the bins 255 - 4 l and the three below
            const int4 c = *reinterpret_cast<const int4 *>(bins + 252 - 4 * lane);
            const int sum = c.x + c.y + c.z + c.w, upto = wave_scan(sum);
            int before = upto - sum, bin = 255 - 4 * lane, count = c.w;
            if (before + count < left) before += count, --bin, count = c.z;
            if (before + count < left) before += count, --bin, count = c.y;
            if (before + count < left) before += count, --bin, count = c.x;
            const int owner = uniform(__builtin_ctzll(__ballot(upto >= left)));
            bin = __builtin_amdgcn_readlane(bin, owner);
            left -= __builtin_amdgcn_readlane(before, owner);
            count = __builtin_amdgcn_readlane(count, owner);
            prefix |= (uint32_t)bin << shift, mask |= ((1u << width) - 1) << shift;
            if (count == left) break;  // all keys with these bits are taken
        }
    }
    for (int i = tid; i < a.first; i += T) out[i] = i;
    for (int i = tid; i < a.recent; i += T) out[a.count - a.recent + i] = hi + i;
    if (none) return;
    if constexpr (T > 64) {
        if (held) {  // by what each wave takes of each T pages, in their order one below the other
            static_assert(kHeld * kWaves <= 64, "one lane for each");
            int before[kHeld];  // in the wave: those with a larger key << 16 | those with the bits
#pragma unroll
            for (int j = 0; j < kHeld; ++j) {
                const uint32_t key = kept[j] & mask;
                const bool there = lo + tid + T * j < hi;
                const unsigned long long m = __ballot(there && key > prefix), e = __ballot(there && key == prefix), below = (1ull << lane) - 1;
                before[j] = __popcll(m & below) << 16 | __popcll(e & below);
                if (lane == 0) space.taken[kWaves * j + wave] = __popcll(m) << 16 | __popcll(e);
            }
            __syncthreads();
            const int mine = lane < kHeld * kWaves ? space.taken[lane] : 0, start = wave_scan(mine) - mine;
#pragma unroll
            for (int j = 0; j < kHeld; ++j) {
                const uint32_t key = kept[j] & mask;
                const int i = lo + tid + T * j, upto = before[j] + __builtin_amdgcn_readlane(start, uniform(kWaves * j + wave));
                const int equals = upto & 0xffff, to = a.first + (upto >> 16) + min(equals, left);
                // below count, but for calls that overlap and share the keys' memory
                if (i < hi && (key > prefix || (key == prefix && equals < left)) && to < a.count) out[to] = i;
            }
            return;
        }
    }
    // place: of the next pick; equals: how many with the bits have been passed
    int place = a.first, equals = 0;
    auto take = [&](int i, uint32_t key) {  // T pages in order, of which the thread has page i
        key &= mask;
        const bool more = i < hi && key > prefix, equal = i < hi && key == prefix;
        const unsigned long long m = __ballot(more), e = __ballot(equal), below = (1ull << lane) - 1;
        int mores = __popcll(m), same = __popcll(e);  // of the wave, then of all
        int m_before = __popcll(m & below), e_before = __popcll(e & below);
        if constexpr (T > 64) {
            __syncthreads();
            if (lane == 0) space.waves[0][wave] = mores << 16 | same;
            __syncthreads();
            mores = same = 0;
#pragma unroll
            for (int x = 0; x < T / 64; ++x) {
                const int s = (int)space.waves[0][x];
                if (x < wave) m_before += s >> 16, e_before += s & 0xffff;
                mores += s >> 16, same += s & 0xffff;
            }
        }
        const int taken = min(equals, left), e_taken = min(equals + e_before, left) - taken;
        const int to = place + m_before + e_taken;  // below count, but for calls that overlap and share the keys' memory
        if ((more || (equal && equals + e_before < left)) && to < a.count) out[to] = i;
        place += mores + min(equals + same, left) - taken;
        equals += same;
    };
    if (held) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if (lo + T * j < hi) take(lo + tid + T * j, kept[j]);
    } else {
        for (int i0 = lo; i0 < hi; i0 += T) take(i0 + tid, key_at(min(i0 + tid, hi - 1)));
    }
}

// Pages that a row at a position sees.
__device__ __forceinline__ int pages_seen(const SelectArgs &a, int pos) { return pos < 0 ? 0 : (pos >> a.shift) + 1; }

// One row and kv head of up to kRowPages pages: scores and picks in one workgroup, the keys in LDS.
template <int D>
__global__ __launch_bounds__(256) void select_row_kernel(SelectArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint32_t keys[];
    __shared__ __attribute__((aligned(16))) uint8_t w[2 * D];
    __shared__ PickSpace<256> space;
    const int t = (int)(blockIdx.x / (uint32_t)a.H), h = (int)blockIdx.x - t * a.H, wave = uniform((int)threadIdx.x >> 6);
    uint32_t page = a.cu ? kNoPage : page_at(a, a.table + t * a.max_pages, 64 * wave);  // beside the length
    const Row row = find_row(a.cu, a.lens, a.B, a.Tq, a.max_pages << a.shift, t);
    if (row.b < 0) return;
    const int seen = pages_seen(a, row.pos);
    if (seen > a.count) {
        const int32_t *table = a.table + row.b * a.max_pages;
        if (a.cu) page = page_at(a, table, 64 * wave);
        auto prepare = [&]() {
            if (wave == 3) query_codes<D>(a, t, h, w);  // the wave with the fewest pages
            __syncthreads();
        };
        score_pages<D, 1>(a, table, h, 64 * wave, 256, seen, 1, page, w, prepare, [&](int, int p, uint4 k) { *reinterpret_cast<uint4 *>(keys + p) = k; });
        __syncthreads();
    }
    pick<256, 1>(a, [&](int i) { return keys[i]; }, seen, a.picks + ((int64_t)t * a.H + h) * a.count, space, threadIdx.x);
}

// The rank-th tile of 16 rows of those of the launch: a sequence that has some, the first
// of them t0 + s, owns the ranks from s / 16 + the number of such sequences before it on
// (room for its rows whatever their number).  n: the tile's rows, 0 if there are none.
struct Tile {
    int b, first, n, pos;  // its first row and that row's position
};
inline int64_t tiles_of(int64_t rows, int64_t B) { return rows / 16 + (B < rows ? B : rows); }
__device__ __forceinline__ Tile find_tile(const SelectArgs &a, int rank) {
    const int lane = threadIdx.x & 63;
    const int64_t room = a.max_pages << a.shift;
    auto length = [&](int b) { return (int)max((int64_t)0, min((int64_t)a.lens[b], room)); };
    if (a.cu == nullptr) return Tile{a.t0 + rank, a.t0 + rank, 1, length(a.t0 + rank) - 1};
    int b = -1, first = 0, end = 0, until = 0, at = 0, floor = 0, before = 0;
    for (int base = 0; base < a.B; base += 64) {
        const int mine = min(base + lane, a.B - 1), to = clamp_row(a.cu[mine + 1], a.Tq);
        const int start = max(floor, wave_scan_max(base + lane < a.B ? clamp_row(a.cu[mine], a.Tq) : 0));
        const int s = clamp_row(start - a.t0, a.rows), e = clamp_row(to - a.t0, a.rows);
        const unsigned long long some = __ballot(base + lane < a.B && e > s);
        const int own = s / 16 + before + __popcll(some & ((1ull << lane) - 1));
        const unsigned long long in = some & __ballot(own <= rank);
        if (in != 0) {  // their ranks rise, so these are the first that have rows
            const int i = 63 - __builtin_clzll(in);
            b = base + i, first = __builtin_amdgcn_readlane(s, i), end = __builtin_amdgcn_readlane(e, i);
            until = __builtin_amdgcn_readlane(to, i), at = __builtin_amdgcn_readlane(own, i);
        }
        before += __popcll(some), floor = __builtin_amdgcn_readlane(start, 63);
        if (in != some || floor - a.t0 >= a.rows) break;
    }
    b = uniform(b);
    if (b < 0) return Tile{0, 0, 0, 0};
    first = uniform(first) + 16 * (rank - uniform(at));
    return Tile{b, a.t0 + first, max(min(16, uniform(end) - first), 0), length(b) - uniform(until) + a.t0 + first};
}

// 16 rows of a sequence and a kv head: the pages' bounds are read once for all of
// them, and each wave picks for one.  510 rows of 8 heads, 40 of up to 938 pages: 17.5 us;
// vector instructions, of the picking for the most part, are issued half of the time.
template <int D>
__global__ __launch_bounds__(1024) void select_tile_kernel(SelectArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint32_t keys[];
    __shared__ __attribute__((aligned(16))) uint8_t w[16 * 2 * D];
    __shared__ PickSpace<64> space[16];
    const int rank = (int)(blockIdx.x / (uint32_t)a.H), h = (int)blockIdx.x - rank * a.H;
    const int wave = uniform((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
    const Tile tile = find_tile(a, rank);
    if (tile.n <= 0) return;
    const int most = pages_seen(a, tile.pos + tile.n - 1);
    if (most > a.count) {
        const int32_t *table = a.table + tile.b * a.max_pages;
        auto prepare = [&]() {
            if (wave < tile.n) query_codes<D>(a, tile.first + wave, h, w + wave * 2 * D);
            __syncthreads();
        };
        score_pages<D, 16>(a, table, h, 64 * wave, 1024, most, tile.n, page_at(a, table, 64 * wave), w, prepare,
                           [&](int r, int p, uint4 k) { *reinterpret_cast<uint4 *>(keys + r * a.pitch + p) = k; });
        __syncthreads();
    }
    if (wave < tile.n)
        pick<64, 16>(a, [&](int i) { return keys[wave * a.pitch + i]; }, pages_seen(a, tile.pos + wave),
                 a.picks + ((int64_t)(tile.first + wave) * a.H + h) * a.count, space[wave], lane);
}

// Scores alone, into memory: 16 rows of a sequence, a kv head and 256 of every
// 256 gridDim.y pages.  48 rows of up to 16,000 tokens, 8 heads of 128 channels, pages of 16:
// 10.5 us for 20 MB, the chain of length, page number and bounds; picking from them 4.4.
template <int D>
__global__ __launch_bounds__(256) void score_kernel(SelectArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t w[16 * 2 * D];
    const int rank = (int)(blockIdx.x / (uint32_t)a.H), h = (int)blockIdx.x - rank * a.H;
    const int wave = uniform((int)threadIdx.x >> 6);
    const int p = 256 * (int)blockIdx.y + 64 * wave;
    uint32_t page = a.cu ? kNoPage : page_at(a, a.table + (a.t0 + rank) * a.max_pages, p);  // beside the length
    const Tile tile = find_tile(a, rank);
    if (tile.n <= 0) return;
    const int most = pages_seen(a, tile.pos + tile.n - 1);
    if (most <= a.count || 256 * (int)blockIdx.y >= most) return;
    const int32_t *table = a.table + tile.b * a.max_pages;
    if (a.cu) page = page_at(a, table, p);
    auto prepare = [&]() {
        for (int r = 3 - wave; r < tile.n; r += 4) query_codes<D>(a, tile.first + r, h, w + r * 2 * D);
        __syncthreads();
    };
    score_pages<D, 16>(a, table, h, p, 256 * (int)gridDim.y, most, tile.n, page, w, prepare, [&](int r, int p, uint4 k) {
        *reinterpret_cast<uint4 *>(a.keys + ((int64_t)(tile.first - a.t0 + r) * a.H + h) * a.pitch + p) = k;
    });
}

template <int T>
__global__ __launch_bounds__(T) void pick_kernel(SelectArgs a) {
    __shared__ PickSpace<T> space;
    const int r = (int)(blockIdx.x / (uint32_t)a.H), h = (int)blockIdx.x - r * a.H, t = a.t0 + r;
    const Row row = find_row(a.cu, a.lens, a.B, a.Tq, a.max_pages << a.shift, t);
    if (row.b < 0) return;
    const uint32_t *keys = a.keys + ((int64_t)r * a.H + h) * a.pitch;
    pick<T, 4>(a, [&](int i) { return keys[i]; }, pages_seen(a, row.pos), a.picks + ((int64_t)t * a.H + h) * a.count, space, threadIdx.x);
}

// Both in one launch, for one new token each: 256 of every 256 gridDim.y pages of a row and kv
// head; the workgroup that finishes last picks, from keys that it reads past its own caches.
template <int D, int kHeld>
__global__ __launch_bounds__(256, 4) void select_parts_kernel(SelectArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t w[2 * D];
    __shared__ PickSpace<256> space;
    __shared__ int arrived;
    if (blockIdx.x == 0 && blockIdx.y == 0) clear_next<256>(a.clear);
    const int t = (int)(blockIdx.x / (uint32_t)a.H), h = (int)blockIdx.x - t * a.H, wave = uniform((int)threadIdx.x >> 6);
    const int p = 256 * (int)blockIdx.y + 64 * wave;
    const int32_t *table = a.table + t * a.max_pages;
    const uint32_t page = page_at(a, table, p);  // beside the length
    const int seen = pages_seen(a, (int)max((int64_t)0, min((int64_t)a.lens[t], a.max_pages << a.shift)) - 1);
    const int parts = seen <= a.count ? 1 : min((int)gridDim.y, (seen + 255) / 256);
    if ((int)blockIdx.y >= parts) return;
    uint32_t *keys = a.keys + (int64_t)blockIdx.x * a.pitch;
    if (seen > a.count) {
        auto prepare = [&]() {
            if (wave == 3) query_codes<D>(a, t, h, w);  // the wave with the fewest pages
            __syncthreads();
        };
        score_pages<D, 1>(a, table, h, p, 256 * (int)gridDim.y, seen, 1, page, w, prepare, [&](int, int i, uint4 k) {
            store_agent(reinterpret_cast<float *>(keys + i), __uint_as_float(k.x), __uint_as_float(k.y));
            store_agent(reinterpret_cast<float *>(keys + i + 2), __uint_as_float(k.z), __uint_as_float(k.w));
        });
        wait_vm0();
        __syncthreads();
        if (parts > 1) {
            if (threadIdx.x == 0) arrived = __hip_atomic_fetch_add(a.counts + blockIdx.x, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            if (uniform(arrived) != parts - 1) return;
        }
    }
    pick<256, kHeld>(a, [&](int i) { return __hip_atomic_load(keys + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }, seen,
              a.picks + (int64_t)blockIdx.x * a.count, space, threadIdx.x);
    if (parts > 1 && threadIdx.x == 0) __hip_atomic_store(a.counts + blockIdx.x, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// -------------------------------------------------------------- attention --
struct BlocksArgs {
    const uint16_t *q;
    const uint8_t *codes;
    const float *scales;
    const int32_t *table, *lens, *cu, *picks;
    uint16_t *o;
    float *part;  // where workgroups leave their parts of an item, ...
    int *counts;  // ... how many have, ...
    int *clear;   // ... and the next call's counters
    int64_t q_ts, q_hs, max_pages, pages;
    int B, Tq, Hq, H, G, shift, count, blocks, parts;  // blocks: of 16 of a kv head's queries
    float scale;                                       // sm_scale log2(e)
};

// The pages that a row reads: entries of its picks, no more than it sees.
__device__ __forceinline__ int entries(const BlocksArgs &a, int pos) { return pos < 0 || a.pages == 0 ? 0 : min(a.count, (pos >> a.shift) + 1); }

// The bits of a step's keys.
template <int kKeys>
struct Bits {
    typedef uint32_t type;
};
template <>
struct Bits<64> {
    typedef uint64_t type;
};

// An item is a row, a kv head and up to 16 of its queries.  Its keys are the picked pages'
// in groups of 16, which lie in one page whatever its size; a wave takes two or four groups
// at a time, a step.  What a wave has of an item: the steps' pages, the codes and scales on
// their way, and the sums.
// The matrix unit's result has 16 columns.  Up to 16 queries have one each (S = 1); up to
// 8 have two, up to 4 four, for S subsets of the keys: column c has query c % (16 / S), and
// of the results of a step's groups that of group c / (16 / S).  So all lanes have scores,
// and each exponential and weight is made once.  The columns of a query have one maximum,
// and their sums are added at the end.  512 rows of 8 kv heads, 40 pages of 32 tokens each,
// e4m3: 4 queries of 64 channels 51 us, 8 of them 59 (S = 1: 70), of 128 channels 110 (115).
template <int D, bool E4M3, int S>
struct Walk {
    static constexpr int kPieces = D / 16, kEach = D / 64;         // 16-byte pieces of a row; of a group, for each lane
    static constexpr int kGroups = S == 4 ? 4 : 2, kSets = S == 1 ? 2 : 1;  // of a step; results, of 4 scores a lane
    static constexpr int kCols = 16 / S, kAhead = 64 / kGroups;     // columns of queries; steps whose pages are looked up together
    static constexpr int kTile = 16 * kGroups * D;                  // bytes of the wave's V tile
    typedef typename Bits<16 * kGroups>::type bits_t;
    const BlocksArgs &a;
    char *turn;  // the wave's V tile in LDS: row r, 16-byte piece c at place c ^ f(r), so that the turning reads spread over the banks
    int lane, quarter, col, own;  // own: the lane's group, where it has one
    // the item: its kv head, the row's position and number of entries; step s has groups g0 + stride s and the next ones
    int h, pos, groups, g0, stride, steps;
    const int32_t *table, *picks;
    int ids, bases;  // of kAhead steps: lane kGroups s + g has of group g of step s the page (-1: none that the row sees) and its first token's position
    uint4 k[kGroups][kEach], v[kGroups][kEach];
    float4 ks[kSets], vs[kSets];
    bf8_t qf[D / 32];
    f4_t acc[D / 16];
    float m, l;

    __device__ __forceinline__ Walk(const BlocksArgs &args, char *lds) : a(args), turn(lds) {
        lane = threadIdx.x & 63, quarter = lane >> 4, col = lane & 15;
        own = col / kCols;
        steps = 0;
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
            for (int c = 0; c < kEach; ++c) k[g][c] = v[g][c] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int x = 0; x < kSets; ++x) ks[x] = vs[x] = make_float4(0, 0, 0, 0);
    }

    __device__ __forceinline__ static int place(int r) { return D == 128 ? (r >> 1) & 7 : (r >> 2) & 3; }

    // The lane's group of the kAhead steps from s0 on, its entry, and what that says once the row is known.
    __device__ __forceinline__ int64_t group(int s0) const {
        return g0 + (int64_t)(s0 + lane / kGroups) * stride + lane % kGroups;
    }
    __device__ __forceinline__ int entry(int s0) const { return picks[min(group(s0) >> (a.shift - 4), (int64_t)a.count - 1)]; }
    __device__ __forceinline__ void look_up(int s0, int pick) {
        const int64_t g = group(s0);
        ids = -1, bases = 0;
        if (g < groups) {
            const int64_t base = ((int64_t)pick << a.shift) + ((g << 4) & ((1 << a.shift) - 1));
            if (pick >= 0 && pick < a.max_pages && base <= pos) {
                const int page = table[pick];
                if ((uint32_t)page < (uint64_t)a.pages) ids = page, bases = (int)base;
            }
        }
    }
    __device__ __forceinline__ int page_of(int s, int g) const { return __builtin_amdgcn_readlane(ids, kGroups * (s % kAhead) + g); }
    __device__ __forceinline__ int base_of(int s, int g) const { return __builtin_amdgcn_readlane(bases, kGroups * (s % kAhead) + g); }

    __device__ __forceinline__ void fetch(int s) {
        const int64_t page_rows = (int64_t)(2 * a.H) << a.shift, to_v = (int64_t)a.H << a.shift;
        // a uniform base and a lane's offset
        uint32_t ko = col * D + quarter * 16, vo = lane * 16, so = 4 * quarter;
        asm("" : "+v"(ko), "+v"(vo), "+v"(so));
        int64_t mine = 0;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const int page = max(page_of(s, g), 0);  // one that does not exist reads page 0: hidden below
            const int64_t at = uniform(page * page_rows + ((int64_t)h << a.shift) + (base_of(s, g) & ((1 << a.shift) - 1)));
            const uint8_t *kp = a.codes + at * D, *vp = kp + to_v * D;
#pragma unroll
            for (int c = 0; c < kEach; ++c) k[g][c] = *reinterpret_cast<const uint4 *>(kp + ko + 64 * c);
#pragma unroll
            for (int c = 0; c < kEach; ++c) v[g][c] = *reinterpret_cast<const uint4 *>(vp + vo + 1024 * c);
            if (S == 1) {
                const float *sp = a.scales + at;
                ks[g % kSets] = *reinterpret_cast<const float4 *>(sp + so);
                vs[g % kSets] = *reinterpret_cast<const float4 *>(sp + to_v + so);
            } else {
                mine = own == g ? at : mine;
            }
        }
        if (S > 1) {
            const float *sp = a.scales + mine + so;
            ks[0] = *reinterpret_cast<const float4 *>(sp);
            vs[0] = *reinterpret_cast<const float4 *>(sp + to_v);
        }
    }

    // the queries t, h G + first .. + rows - 1, as B operands with the channels in the order of K's pieces
    __device__ __forceinline__ void queries(int t, int first, int rows) {
        const uint16_t *qp = a.q + (int64_t)t * a.q_ts + (int64_t)(h * a.G + first + min(col % kCols, rows - 1)) * a.q_hs;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) qf[i] = *reinterpret_cast<const bf8_t *>(qp + 16 * (quarter + 4 * (i / 2)) + 8 * (i & 1));
    }

    // The columns of a query: the largest, the sum.
    __device__ __forceinline__ static float max_columns(float x) {
        if (S > 1) x = fmaxf(x, dpp_f32<0x128>(x));  // row_ror 8
        if (S > 2) x = fmaxf(x, dpp_f32<0x124>(x));  // row_ror 4
        return x;
    }
    __device__ __forceinline__ static float sum_columns(float x) {
        if (S > 1) x += dpp_f32<0x128>(x);
        if (S > 2) x += dpp_f32<0x124>(x);
        return x;
    }

    // A step; masked: of some group not all 16 keys are seen.  What is hidden is
    // hidden from all columns, which are queries of one token: its values are taken as zeros.
    template <bool kMasked>
    __device__ __forceinline__ void step(int s, bits_t seen) {
#pragma unroll
        for (int c = 0; c < kGroups * kEach; ++c) {
            const int r = lane / kPieces + c * (64 / kPieces);
            uint4 &w = v[c / kEach][c % kEach];
            if (E4M3 && kMasked && !((seen >> r) & 1)) w = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(turn + r * D + (((lane % kPieces) ^ place(r)) << 4)) = w;
        }
        float kc[kSets][4], vc[kSets][4];
#pragma unroll
        for (int x = 0; x < kSets; ++x) {
            kc[x][0] = ks[x].x * a.scale, kc[x][1] = ks[x].y * a.scale, kc[x][2] = ks[x].z * a.scale, kc[x][3] = ks[x].w * a.scale;
            vc[x][0] = vs[x].x, vc[x][1] = vs[x].y, vc[x][2] = vs[x].z, vc[x][3] = vs[x].w;
            // copies, so that the next step's loads are not waited for at the end of this one
#pragma unroll
            for (int r = 0; r < 4; ++r) asm volatile("" : "+v"(vc[x][r]));
        }
        f4_t sc[kSets];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            f4_t x = {};
#pragma unroll
            for (int c = 0; c < kEach; ++c) {
                const uint4 w = k[g][c];
                x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode8<E4M3>(w.x, w.y), qf[2 * c], x, 0, 0, 0);
                x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode8<E4M3>(w.z, w.w), qf[2 * c + 1], x, 0, 0, 0);
            }
            if (S == 1 || g == 0)
                sc[g % kSets] = x;
            else
#pragma unroll
                for (int r = 0; r < 4; ++r) sc[0][r] = own == g ? x[r] : sc[0][r];
        }
        ahead(s);
        bool hid[kSets][4];
        const uint32_t vis = (uint32_t)(seen >> (S == 1 ? 4 * quarter : 16 * own + 4 * quarter));
#pragma unroll
        for (int x = 0; x < kSets; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                sc[x][r] *= kc[x][r];
                hid[x][r] = kMasked && !((vis >> (16 * x + r)) & 1);
                if (kMasked) sc[x][r] = hid[x][r] ? kNegInf : sc[x][r];
            }
        float top = sc[0][0];
#pragma unroll
        for (int i = 1; i < 4 * kSets; ++i) top = fmaxf(top, sc[i / 4][i % 4]);
        if (__any(top > m + kSlack)) {
            const float m1 = fmaxf(m, max_columns(max_quarters(top)));
            const float f = m1 == kNegInf ? 1.0f : exp2_fast(m - m1);
            m = m1;
            l *= f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) acc[i] *= f;
        }
        const float ms = m == kNegInf ? 0.0f : m;
        // a weight is the sum of two bf16: its rounding and the rounding of what that leaves
        uint32_t p[2 * kSets], pr[2 * kSets];
#pragma unroll
        for (int i = 0; i < 2 * kSets; ++i) {
            float w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int x = i / 2, r = 2 * (i & 1) + e;
                const float pe = exp2_fast(sc[x][r] - ms);
                l += pe;
                w[e] = hid[x][r] ? 0.0f : pe * vc[x][r];  // a hidden key's scale may be anything
            }
            p[i] = pack_bf16(w[0], w[1]);
            pr[i] = pack_bf16(w[0] - __uint_as_float(p[i] << 16), w[1] - __uint_as_float(p[i] & 0xffff0000u));
        }
        // The products of 32 keys and the weights, zeros in the columns of other groups.  With four
        // groups half of the columns would be idle in each: they take what the first rounding left of
        // the weights in the other half.
        constexpr int kPairs = kGroups / 2, kTerms = S == 4 ? 1 : 2;
        bf8_t pf[kPairs][kTerms];
        auto operand = [&](uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
            return __builtin_bit_cast(bf8_t, i4_t{(int)w0, (int)w1, (int)w2, (int)w3});
        };
        const bool even = (own & 1) == 0;
        if constexpr (S == 1) {
            pf[0][0] = operand(p[0], p[1], p[2], p[3]), pf[0][1] = operand(pr[0], pr[1], pr[2], pr[3]);
        } else if constexpr (S == 2) {
            pf[0][0] = operand(even ? p[0] : 0, even ? p[1] : 0, even ? 0 : p[0], even ? 0 : p[1]);
            pf[0][1] = operand(even ? pr[0] : 0, even ? pr[1] : 0, even ? 0 : pr[0], even ? 0 : pr[1]);
        } else {
            const uint32_t r0 = dpp_u32<0x128>(pr[0]), r1 = dpp_u32<0x128>(pr[1]);  // row_ror 8
            const bool low = own < 2;
            const uint32_t x0 = low ? p[0] : r0, x1 = low ? p[1] : r1, y0 = low ? r0 : p[0], y1 = low ? r1 : p[1];
            pf[0][0] = operand(even ? x0 : 0, even ? x1 : 0, even ? 0 : x0, even ? 0 : x1);
            pf[1][0] = operand(even ? y0 : 0, even ? y1 : 0, even ? 0 : y0, even ? 0 : y1);
        }
        // V^T: keys 4 quarter + 0..3 and 16 + 4 quarter + 0..3 of 16 channels
        const int vkey = 4 * quarter + ((col >> 1) & 3) + 16 * (col >> 3);
        int xv = place(vkey) << 4;
        asm("" : "+v"(xv));  // 8 addresses made anew in each step, not kept
        const char *from = turn + vkey * D + (col & 1) * 8;
#pragma unroll
        for (int j = 0; j < kPairs; ++j)
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const i2_t w = __builtin_amdgcn_ds_read_tr8_b64_v2i32((LDS_AS i2_t *)(from + 32 * j * D + ((i << 4) ^ xv)));
                const bf8_t vf = decode8<E4M3>((uint32_t)w[0], (uint32_t)w[1]);
#pragma unroll
                for (int x = 0; x < kTerms; ++x) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[j][x], acc[i], 0, 0, 0);
            }
    }

    // The loads of the step behind s; behind the last the last one's again: without a branch
    // they land where the others were, with one the compiler keeps both and copies (80 us
    // where 97 were measured: 510 rows of 64 channels, 40 pages of 32 tokens each).
    __device__ __forceinline__ void ahead(int s) {
        const int n = min(s + 1, steps - 1);
        if (n > s && n % kAhead == 0) look_up(n, entry(n));
        fetch(n);
    }

    // Of a step's keys those that the row sees, as bits.
    __device__ __forceinline__ bits_t seen_of(int s) const {
        auto low_bits = [](int n) { return n <= 0 ? 0u : n >= 16 ? 0xffffu : (1u << n) - 1; };
        bits_t seen = 0;
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
            seen |= (bits_t)(page_of(s, g) < 0 ? 0u : low_bits(pos + 1 - base_of(s, g))) << (16 * g);
        return seen;
    }

    // All steps, the first of which is on its way; the sums of a lane's column are then complete.
    __device__ __forceinline__ void run() {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) acc[i] = f4_t{};
        m = kNegInf, l = 0.0f;
        for (int s = 0; s < steps; ++s) {
            bits_t seen = seen_of(s);
            while (seen == ~bits_t{0}) {  // a loop of its own, whose registers need no copies
                step<false>(s, seen);
                seen = ++s < steps ? seen_of(s) : 0;
            }
            if (s >= steps) break;
            if (seen != 0)
                step<true>(s, seen);
            else
                ahead(s);
        }
        l = sum_columns(sum_quarters(l));
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][r] = sum_columns(acc[i][r]);
    }
};

// Many items: one for each wave, the same kv head of 4 neighbouring rows in a workgroup.
// With 64 channels four waves of a SIMD share the registers (51 us where three took 54), of
// which up to three are spilled with 4 queries in e4m3 and with more than 8.
// 510 rows of 4 queries of 8 heads of 64 channels, 40 pages of 32 tokens, e4m3: 55 us; vector
// instructions take 63 % of the time and the matrix unit 18 %, and they hardly overlap.
template <int D, bool E4M3, int S>
__global__ __launch_bounds__(256, D == 64 ? 4 : 2) void attn_blocks_many_kernel(BlocksArgs a) {
    typedef Walk<D, E4M3, S> W;
    __shared__ __attribute__((aligned(1024))) char lds[4 * W::kTile];
    const int wave = uniform((int)threadIdx.x >> 6), per_row = a.H * a.blocks;
    const int t = (int)(blockIdx.x / (uint32_t)per_row) * 4 + wave, hb = (int)(blockIdx.x % (uint32_t)per_row);
    if (t >= a.Tq) return;
    W w(a, lds + wave * W::kTile);
    w.h = hb / a.blocks;
    const int first = (hb - w.h * a.blocks) * 16, rows = min(16, a.G - first);
    w.picks = a.picks + ((int64_t)t * a.H + w.h) * a.count, w.g0 = 0, w.stride = W::kGroups;
    const int pick = w.entry(0);  // on its way while the row is looked for
    const Row row = find_row(a.cu, a.lens, a.B, a.Tq, a.max_pages << a.shift, t);
    if (row.b < 0) return;
    w.pos = row.pos, w.groups = entries(a, row.pos) << (a.shift - 4), w.steps = (w.groups + W::kGroups - 1) / W::kGroups;
    w.table = a.table + row.b * a.max_pages;
    w.look_up(0, pick);
    w.queries(t, first, rows);
    if (w.steps > 0) w.fetch(0);
    w.run();
    if (w.col >= rows) return;
    uint16_t *op = a.o + ((int64_t)t * a.Hq + w.h * a.G + first + w.col) * D + 4 * w.quarter;
    const float inv = w.l == 0.0f ? 0.0f : 1.0f / w.l;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
        *reinterpret_cast<uint2 *>(op + 16 * i) =
            make_uint2(pack_bf16(w.acc[i][0] * inv, w.acc[i][1] * inv), pack_bf16(w.acc[i][2] * inv, w.acc[i][3] * inv));
}

// Few items: the 4 waves of a workgroup, and `parts` workgroups, take an item's steps in
// turn; they are joined in LDS, and over the parts by the workgroup that finishes last
// (qw3_attn_dev.h).  48 rows of 8 heads, 64 pages of 16 tokens of 128 channels: 20 us for 62
// MB; a CU reads some 30 bytes a ns, and of 384 items many have to share one.
template <int D, bool E4M3, int S>
__global__ __launch_bounds__(256, 2) void attn_blocks_few_kernel(BlocksArgs a) {
    typedef Walk<D, E4M3, S> Wave;
    constexpr int R = 16, W = 4, kPad = D + 4;
    constexpr int kTurn = W * Wave::kTile, kJoin = W * R * kPad * 4;
    __shared__ __attribute__((aligned(1024))) char lds[kTurn > kJoin ? kTurn : kJoin];
    __shared__ float stat[2][W][R];
    __shared__ int arrived;
    const int tid = threadIdx.x, wave = uniform(tid >> 6), per_row = a.H * a.blocks;
    if (a.parts > 1 && blockIdx.x == 0) clear_next<256>(a.clear);
    const int item = (int)(blockIdx.x / (uint32_t)a.parts), part = (int)blockIdx.x - item * a.parts;
    const int t = (int)((uint32_t)item / (uint32_t)per_row), hb = item - t * per_row;
    Wave w(a, lds + wave * Wave::kTile);
    w.h = hb / a.blocks;
    const int first = (hb - w.h * a.blocks) * R, rows = min(R, a.G - first);
    w.picks = a.picks + ((int64_t)t * a.H + w.h) * a.count;
    w.g0 = Wave::kGroups * (part * W + wave), w.stride = Wave::kGroups * W * a.parts;
    const int pick = w.entry(0);  // on its way while the row is looked for
    w.queries(t, first, rows);
    const Row row = find_row(a.cu, a.lens, a.B, a.Tq, a.max_pages << a.shift, t);
    if (row.b < 0) return;  // all parts
    w.pos = row.pos, w.groups = entries(a, row.pos) << (a.shift - 4);
    w.steps = w.g0 < w.groups ? (w.groups - w.g0 + w.stride - 1) / w.stride : 0;
    w.table = a.table + row.b * a.max_pages;
    if (w.steps > 0) w.look_up(0, pick);
    if (w.steps > 0) w.fetch(0);
    w.run();

    uint16_t *op = a.o + ((int64_t)t * a.Hq + w.h * a.G + first) * D;
    float *join = reinterpret_cast<float *>(lds);
    float *out = a.part + (int64_t)blockIdx.x * (R * (D + 2));
    if (w.quarter == 0) stat[0][wave][w.col] = w.m, stat[1][wave][w.col] = w.l;
    lds_barrier();  // the turning tiles are read
#pragma unroll
    for (int i = 0; i < D / 16; ++i) *reinterpret_cast<f4_t *>(join + (wave * R + w.col) * kPad + 16 * i + 4 * w.quarter) = w.acc[i];
    lds_barrier();
    for (int e = tid; e < rows * D / 2; e += 256) {
        const int r = e / (D / 2), c = 2 * (e % (D / 2));
        float mm = kNegInf;
#pragma unroll
        for (int x = 0; x < W; ++x) mm = fmaxf(mm, stat[0][x][r]);
        float ll = 0.0f;
        f2_t sum = {};
#pragma unroll
        for (int x = 0; x < W; ++x) {
            const float f = stat[0][x][r] == kNegInf ? 0.0f : exp2_fast(stat[0][x][r] - mm);
            ll += f * stat[1][x][r];
            sum += f * *reinterpret_cast<const f2_t *>(join + (x * R + r) * kPad + c);
        }
        if (a.parts == 1) {
            const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
            *reinterpret_cast<uint32_t *>(op + r * D + c) = pack_bf16(sum[0] * inv, sum[1] * inv);
        } else {
            store_agent(out + 2 * R + r * D + c, sum[0], sum[1]);
            if (c == 0) store_agent(out + 2 * r, mm, ll);
        }
    }
    if (a.parts == 1) return;
    wait_vm0();
    __syncthreads();
    if (tid == 0) arrived = __hip_atomic_fetch_add(a.counts + item, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (uniform(arrived) != a.parts - 1) return;
    const float *parts0 = a.part + (int64_t)item * a.parts * (R * (D + 2));
    auto slot_of = [&](int g) -> const float * { return parts0 + (int64_t)g * (R * (D + 2)); };
    auto row_out = [&](int r) { return op + r * D; };
    if (rows <= R / 2)
        join_rows<R, D, R / 8>(slot_of, 0, a.parts - 1, rows, row_out);
    else
        join_rows<R, D, R / 4>(slot_of, 0, a.parts - 1, rows, row_out);
    if (tid == 0) __hip_atomic_store(a.counts + item, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <int D, bool E4M3, int S>
qw3_status launch_many(const BlocksArgs &a, hipStream_t stream) {
    const int64_t wgs = ceil_div(a.Tq, 4) * a.H * a.blocks;
    hipLaunchKernelGGL((attn_blocks_many_kernel<D, E4M3, S>), dim3((unsigned)wgs), dim3(256), 0, stream, a);
    return check_launch();
}
template <int D, bool E4M3, int S>
qw3_status launch_few(const BlocksArgs &a, int64_t items, hipStream_t stream) {
    hipLaunchKernelGGL((attn_blocks_few_kernel<D, E4M3, S>), dim3((unsigned)(items * a.parts)), dim3(256), 0, stream, a);
    return check_launch();
}

template <int D, bool E4M3>
qw3_status launch_blocks(BlocksArgs a, hipStream_t stream) {
    int cus = 0;
    qw3_status st = cu_count(&cus);
    if (st != QW3_OK) return st;
    const int64_t items = (int64_t)a.Tq * a.H * a.blocks;
    const int subsets = a.G <= 4 ? 4 : a.G <= 8 ? 2 : 1;
    if (items >= 8 * (int64_t)cus)  // an item for each wave fills the card
        return subsets == 4   ? launch_many<D, E4M3, 4>(a, stream)
               : subsets == 2 ? launch_many<D, E4M3, 2>(a, stream)
                              : launch_many<D, E4M3, 1>(a, stream);
    // An item of n units of 128 keys in parts of u units takes u + 0.14 n / u, as in
    // qattn_cache: least at u = sqrt(0.14 n); and no more parts than the CUs have room for,
    // two workgroups each.  One row of 8 kv heads, 64 pages of 64 tokens, with 1, 4, 8, 16, 32
    // parts: 49, 19, 13.5, 12.5, 14 us; 48 rows of 8, 64 pages of 16, with 1, 2, 4: 22, 26, 31.
    const int64_t entries = a.count < a.max_pages ? a.count : a.max_pages;
    const float units = (float)((entries << a.shift) / 128 + 1);
    const int most = (int)(units / __builtin_sqrtf(0.14f * units));
    const int64_t room = items < 2 * (int64_t)cus ? 2 * (int64_t)cus / items : 1;
    a.parts = (int)(room < most ? room : most);
    if (a.parts < 1 || items > kCounts) a.parts = 1;
    Scratch ws;
    if (a.parts > 1) {
        st = workspace(stream, (size_t)(items * a.parts) * 16 * (D + 2) * sizeof(float), &ws);
        if (st != QW3_OK) return st;
        a.part = static_cast<float *>(ws.ptr);
        st = counters(stream, (int)items, &a.counts, &a.clear);
        if (st != QW3_OK) return st;
    }
    // Workgroups that are all on the card at once wait for memory, and gain nothing from fewer
    // instructions: 48 rows of 8 heads, 64 pages of 16 tokens of 128 channels, S = 1, 2, 4: 19, 20,
    // 21 us; 500 rows of 2 heads, 100 pages of 32 tokens of 64 channels: 58, 50, 45.
    if (items <= 2 * (int64_t)cus || subsets == 1) return launch_few<D, E4M3, 1>(a, items, stream);
    return subsets == 4 ? launch_few<D, E4M3, 4>(a, items, stream) : launch_few<D, E4M3, 2>(a, items, stream);
}

constexpr int64_t kTileKeys = 32768;              // words of LDS for the keys of 16 rows
constexpr int64_t kKeyBytes = int64_t(64) << 20;  // of keys in memory at a time
constexpr int64_t kRowPages = 256, kPartPages = 2048;

// One CU reads some 30 bytes of bounds a ns, 512 pages of 128 channels in 4.5 us.  So a row's
// pages are read by one workgroup only where a table has few; else by as many as there are
// pages for, through memory, of which the last picks; or a second launch, where there are more
// workgroups than counters, more keys than 256 threads keep, or several rows of a sequence.
// 64 pages for one row of 8 kv heads, tables of 250, 512, 1024, 2048, 4096: by one workgroup 7.8,
// 11.5, 19.7, 34.9 us, by the last 9.9 (260), 9.9, 10.2, 12.2, 16.4, by a second launch 12.1, 12.2,
// 11.9, 12.7, 13.6.  48 rows, 250, 512, 1024, 2048: by one 10.0, 17.4, 28.5, by the last 12.4, 17.8,
// 29.3, 51.3, by a second launch 14.1, 21.1, 31.1, 56.5; 17 to 16,000 tokens each in pages of 16, where
// the longest are waited for: 19.9, 15.4, 15.8.
// The host knows the table's width alone.  Where it is more than the rows see: 24 pages for one row
// over 1000 tokens in pages of 16, tables of 63 to 250 pages 6.5 us, 257 to 1024 8.1, 2048 8.8, 2049 to
// 8192 9.5; 16 such rows 6.6, 8.3 (512), 9.2 (2048), 10.7 (8192).
template <int D>
qw3_status launch_select(SelectArgs a, hipStream_t stream) {
    int cus = 0;
    qw3_status st = cu_count(&cus);
    if (st != QW3_OK) return st;
    a.pitch = (int)(ceil_div(a.max_pages, 16) * 16 + 4);  // rows of the keys begin in different banks
    if (a.cu && a.Tq >= 4 * (int64_t)a.B && 16 * a.pitch <= kTileKeys) {
        a.rows = a.Tq;
        hipLaunchKernelGGL((select_tile_kernel<D>), dim3((unsigned)(tiles_of(a.Tq, a.B) * a.H)), dim3(1024), 16 * a.pitch * 4, stream, a);
        return check_launch();
    }
    if (a.max_pages <= kRowPages) {
        hipLaunchKernelGGL((select_row_kernel<D>), dim3((unsigned)(a.Tq * a.H)), dim3(256), a.pitch * 4, stream, a);
        return check_launch();
    }
    int64_t rows = kKeyBytes / (4 * (int64_t)a.pitch * a.H);
    rows = rows < 16 ? 16 : rows;
    rows = rows < a.Tq ? rows : a.Tq;
    Scratch ws;
    st = workspace(stream, (size_t)(rows * a.H * a.pitch) * 4, &ws);
    if (st != QW3_OK) return st;
    a.keys = static_cast<uint32_t *>(ws.ptr);
    int64_t some = ceil_div(a.max_pages, 256);  // workgroups of a tile
    some = some < 64 ? some : 64;
    if (!a.cu && a.max_pages <= kPartPages && a.Tq * (int64_t)a.H <= kCounts) {
        st = counters(stream, a.Tq * a.H, &a.counts, &a.clear);
        if (st != QW3_OK) return st;
        const auto kernel = a.max_pages <= 1024 ? select_parts_kernel<D, 4> : select_parts_kernel<D, 8>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)(a.Tq * a.H), (unsigned)some), dim3(256), 0, stream, a);
        return check_launch();
    }
    for (int64_t t = 0; t < a.Tq; t += rows) {
        a.t0 = (int)t, a.rows = (int)(rows < a.Tq - t ? rows : a.Tq - t);
        // tiles of these rows alone, so that the work grows with the rows whatever the batches: a chunk of
        // 30,000 rows over 8192 pages, 8 heads, is 118 batches
        const int64_t tiles = a.cu ? tiles_of(a.rows, a.B) : a.rows;
        hipLaunchKernelGGL((score_kernel<D>), dim3((unsigned)(tiles * a.H), (unsigned)some), dim3(256), 0, stream, a);
        if ((int64_t)a.rows * a.H >= cus)
            hipLaunchKernelGGL((pick_kernel<256>), dim3((unsigned)(a.rows * a.H)), dim3(256), 0, stream, a);
        else
            hipLaunchKernelGGL((pick_kernel<1024>), dim3((unsigned)(a.rows * a.H)), dim3(1024), 0, stream, a);
    }
    return check_launch();
}

// What the three calls check of sequences; *shift = log2(page_size).
qw3_status check_sequences(int64_t B, int64_t max_pages, int64_t Tq, bool starts, int64_t H, int64_t D, int64_t pages,
                           int64_t page_size, int *shift) {
    const qw3_status st = check_cache(QW3_CODES_INT8, H, D, pages, page_size, shift);
    if (st != QW3_OK) return st;
    if (B < 0 || B > QW3_MAX_SEQS || Tq < 0 || Tq > QW3_MAX_TOKENS || max_pages < 0 || (!starts && Tq != B)) return QW3_ERR_SHAPE;
    return max_pages > (int64_t(1) << 30) / page_size ? QW3_ERR_SHAPE : QW3_OK;
}

qw3_status check_picks(int64_t Tq, int64_t Hq, int64_t H, int64_t count, int64_t q_ts, int64_t q_hs) {
    if (Hq < 1 || Hq % H != 0 || Hq > QW3_MAX_HEADS || count < 1 || count > QW3_MAX_PICKS) return QW3_ERR_SHAPE;
    if ((Tq + 4) * H * ceil_div(Hq / H, 16) >= 4 * kMaxGroups) return QW3_ERR_SHAPE;  // a wave for each item
    return strides_ok(q_ts, q_hs, int64_t(1) << 32) ? QW3_OK : QW3_ERR_SHAPE;
}

}  // namespace

extern "C" {

qw3_status qcache_bounds(const void *codes, const float *scales, int32_t code_type, const int32_t *block_table,
                         const int32_t *lens, const int32_t *cu_q, int8_t *bounds, float *bound_scales, int64_t B,
                         int64_t max_pages, int64_t Tq, int64_t H, int64_t D, int64_t pages, int64_t page_size,
                         void *hip_stream) {
    int shift = 0;
    if (code_type != QW3_CODES_INT8 && code_type != QW3_CODES_E4M3) return QW3_ERR_SHAPE;
    const qw3_status st = check_sequences(B, max_pages, Tq, cu_q != nullptr, H, D, pages, page_size, &shift);
    if (st != QW3_OK) return st;
    const int64_t items = cu_q ? (Tq >> shift) + 2 * B : B;
    if (items * H >= 4 * kMaxGroups) return QW3_ERR_SHAPE;
    if (B == 0 || Tq == 0 || max_pages == 0 || pages == 0) return QW3_OK;
    if (!codes || !scales || !block_table || !lens || !bounds || !bound_scales) return QW3_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(block_table, 4) || !aligned(lens, 4) || !aligned(cu_q, 4) ||
        !aligned(bounds, 16) || !aligned(bound_scales, 4))
        return QW3_ERR_ALIGN;
    BoundsArgs a{};
    a.codes = static_cast<const uint8_t *>(codes), a.scales = scales, a.table = block_table, a.lens = lens, a.cu = cu_q;
    a.bounds = bounds, a.steps = bound_scales, a.B = (int)B, a.Tq = (int)Tq, a.H = (int)H, a.shift = shift;
    a.items = (int)items, a.max_pages = max_pages, a.pages = pages;
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)ceil_div(items * H, 4)), dim3(256), 0, (hipStream_t)hip_stream, a);
    };
    if (D == 128)
        code_type == QW3_CODES_E4M3 ? run(bounds_kernel<128, true>) : run(bounds_kernel<128, false>);
    else
        code_type == QW3_CODES_E4M3 ? run(bounds_kernel<64, true>) : run(bounds_kernel<64, false>);
    return check_launch();
}

qw3_status qblock_select(const uint16_t *q, const int8_t *bounds, const float *bound_scales, const int32_t *block_table,
                         const int32_t *lens, const int32_t *cu_q, int32_t *picks, int64_t B, int64_t max_pages, int64_t Tq,
                         int64_t Hq, int64_t H, int64_t D, int64_t pages, int64_t page_size, int64_t count, int64_t first,
                         int64_t recent, int64_t q_ts, int64_t q_hs, void *hip_stream) {
    int shift = 0;
    qw3_status st = check_sequences(B, max_pages, Tq, cu_q != nullptr, H, D, pages, page_size, &shift);
    if (st != QW3_OK) return st;
    st = check_picks(Tq, Hq, H, count, q_ts, q_hs);
    if (st != QW3_OK) return st;
    if (first < 0 || recent < 1 || first > count || recent > count - first) return QW3_ERR_SHAPE;
    if ((Tq + B) * H >= kMaxGroups / 4) return QW3_ERR_SHAPE;  // of workgroups of 1024 threads
    if (B == 0 || Tq == 0) return QW3_OK;
    if (!q || !lens || !picks || (max_pages > 0 && !block_table) || (pages > 0 && (!bounds || !bound_scales))) return QW3_ERR_NULL;
    if (!aligned(q, 16) || !aligned(bounds, 16) || !aligned(bound_scales, 4) || !aligned(block_table, 4) || !aligned(lens, 4) ||
        !aligned(cu_q, 4) || !aligned(picks, 4) || q_ts % 8 || q_hs % 8)
        return QW3_ERR_ALIGN;
    SelectArgs a{};
    a.q = q, a.bounds = bounds, a.steps = bound_scales, a.table = block_table, a.lens = lens, a.cu = cu_q, a.picks = picks;
    a.q_ts = q_ts, a.q_hs = q_hs, a.max_pages = max_pages, a.pages = pages, a.B = (int)B, a.Tq = (int)Tq, a.H = (int)H;
    a.G = (int)(Hq / H), a.shift = shift, a.count = (int)count, a.first = (int)first, a.recent = (int)recent;
    return D == 128 ? launch_select<128>(a, (hipStream_t)hip_stream) : launch_select<64>(a, (hipStream_t)hip_stream);
}

qw3_status qattn_blocks(const uint16_t *q, const void *codes, const float *scales, int32_t code_type,
                        const int32_t *block_table, const int32_t *lens, const int32_t *cu_q, const int32_t *picks,
                        uint16_t *out, int64_t B, int64_t max_pages, int64_t Tq, int64_t Hq, int64_t H, int64_t D,
                        int64_t pages, int64_t page_size, int64_t count, int64_t q_ts, int64_t q_hs, float sm_scale,
                        void *hip_stream) {
    int shift = 0;
    if (code_type != QW3_CODES_INT8 && code_type != QW3_CODES_E4M3) return QW3_ERR_SHAPE;
    qw3_status st = check_sequences(B, max_pages, Tq, cu_q != nullptr, H, D, pages, page_size, &shift);
    if (st != QW3_OK) return st;
    st = check_picks(Tq, Hq, H, count, q_ts, q_hs);
    if (st != QW3_OK) return st;
    if (count > (int64_t(1) << 30) / page_size || !(sm_scale > 0.0f && sm_scale < __builtin_huge_valf())) return QW3_ERR_SHAPE;
    if (B == 0 || Tq == 0) return QW3_OK;
    if (!q || !lens || !picks || !out || (max_pages > 0 && !block_table) || (pages > 0 && (!codes || !scales))) return QW3_ERR_NULL;
    if (!aligned(q, 16) || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(block_table, 4) || !aligned(lens, 4) ||
        !aligned(cu_q, 4) || !aligned(picks, 4) || !aligned(out, 16) || q_ts % 8 || q_hs % 8)
        return QW3_ERR_ALIGN;
    BlocksArgs a{};
    a.q = q, a.codes = static_cast<const uint8_t *>(codes), a.scales = scales, a.table = block_table, a.lens = lens;
    a.cu = cu_q, a.picks = picks, a.o = out, a.q_ts = q_ts, a.q_hs = q_hs, a.max_pages = max_pages, a.pages = pages;
    a.B = (int)B, a.Tq = (int)Tq, a.Hq = (int)Hq, a.H = (int)H, a.G = (int)(Hq / H), a.shift = shift, a.count = (int)count;
    a.blocks = (int)ceil_div(Hq / H, 16), a.scale = sm_scale * 1.44269504088896341f;
    const hipStream_t stream = (hipStream_t)hip_stream;
    if (D == 128) return code_type == QW3_CODES_E4M3 ? launch_blocks<128, true>(a, stream) : launch_blocks<128, false>(a, stream);
    return code_type == QW3_CODES_E4M3 ? launch_blocks<64, true>(a, stream) : launch_blocks<64, false>(a, stream);
}

}  // extern "C"
