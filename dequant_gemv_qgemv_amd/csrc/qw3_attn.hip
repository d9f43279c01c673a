// Attention between the products: qattn_prompt (whole prompts) and qattn_cache
// (new or drafted tokens over the quantised cache).  C ABI in include/qw3.h.
//
// Both compute, for a query row with the visible keys V,
//   o = sum_{j in V} p_j v_j / sum_{j in V} p_j,   p_j = 2^(c q.k_j - m),
// c = sm_scale log2(e), m a running maximum over the keys read so far: one
// pass over the keys, the sums rescaled by 2^(m - m') when m grows to m'.
// Scores, m, the sum of p and the weighted sum of v stay in fp32; only the
// weights of the v_j are rounded, to bf16 for the matrix unit (at most 2^-8 of a
// term, the rounding of the output itself), and with few rows to two bf16 each.
//
// Orientation.  The matrix unit computes S^T = K Q^T, so a query row is a
// column of the result: one lane holds many keys of one row, the row's maximum
// and sum are mostly in-lane, and S^T's registers are, as they lie, the B
// operand of O^T = V^T P^T once V's rows are taken in the same order.  The
// rescale factor of a row is then one value per lane.  V^T comes from row-major
// tiles in LDS through the transposing LDS reads.
#include "qw3_attn_dev.h"
#include "qw3_host.h"

#include <vector>

using namespace qw3_shared;

namespace {

// A buffer descriptor over `bytes` bytes at p (both the same in every lane);
// reads past the end give zeros.
__device__ __forceinline__ i4_t descriptor(const void *p, uint32_t bytes) {
    const int64_t a = uniform(reinterpret_cast<int64_t>(p));
    return i4_t{(int)(uint32_t)a, (int)((uint32_t)((uint64_t)a >> 32) & 0xffffu), uniform((int)bytes), 0x00020000};
}

// 64 lanes x 16 bytes from memory straight into LDS: lane i's bytes land at
// byte address lds + 16 i.  The caller waits for vmcnt before it reads them.  In
// asm because the compiler, which cannot tell the buffers of a ring apart, would
// wait for the newest load before every LDS read.  M0 carries the address;
// nothing else in these kernels uses it.
__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t voffset, i4_t desc) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voffset), "s"(desc)
                 : "memory");
}

__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return (uint32_t)uniform((int)reinterpret_cast<uintptr_t>((LDS_AS const char *)p));
}

// Until at most N of the wave's loads are on the way, then for the other waves.
template <int N>
__device__ __forceinline__ void wait_loads_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// x plus the two bf16 of p.
__device__ __forceinline__ float add_pair(uint32_t p, float x) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf2_t, p), __builtin_bit_cast(bf2_t, 0x3f803f80u), x, false);
}

// What the matrix-bound kernels cost.  On this card matrix and vector
// instructions of a SIMD hardly run at the same time: for two waves of a SIMD,
// 16 32x32x16 products each take 608 ns alone, 192 fma 449 ns alone, both 900 ns
// mixed in one wave and 1041 ns from two.  So a kernel's time is the sum of the
// two, and what counts is the number of vector instructions beside a product,
// not their order (interleaving them by hand measured within 2 %).

// ================================================================= prompt ==
struct PromptArgs {
    const uint16_t *q, *k, *v;
    uint16_t *o;
    const int32_t *cu_q, *cu_k;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;  // strides in elements
    int B, Tq, Tk, Hq, H, tiles;
    float scale;  // sm_scale log2(e)
    int slices;   // with SPLIT: workgroups for one tile's keys, at most, ...
    float *part;  // ... where they leave their parts, and ...
    int *counts;  // ... how many have
    int *clear;   // the next call's counters
};

constexpr int kKeys = 64;  // of a tile

// Slices of a tile's keys.  A workgroup takes 0.6 us for a tile of keys, adding a
// part costs about twice that: slices of u of n tiles are worth it from u = sqrt(2
// n) on, and from 16 tiles on.  Measured whole, and with factors 0.3, 1 and 2: 1 row
// of 8 heads of 128 channels against 6000 keys 59, 24, 20 and 20 us, 100 rows of 64
// heads 61, 39, 39, 39; but against 700 keys 13.4 us whole, 16.6 in slices.
constexpr float kSliceJoin = 2.0f;
constexpr int kSliceLeast = 16;

// Hidden values that are not numbers.  The tiles multiply hidden keys by p = 0,
// which is not 0 where a hidden value row holds an infinity or NaN.  A row whose
// outputs come out non-finite is computed again from the keys it sees alone, but
// only if such a value lies among the hidden keys of its tiles (at most 94 behind
// its last): otherwise what it sees made it so, and it is right as it is.  8192
// tokens of 64 heads, NaN in a value of one kv head: as without (1.0 ms) for most
// tokens, 14 ms for the last one's (a wave computes its 31 other rows one by one).

// The last of the keys first..end - 1 whose value row is not finite, or -1.
template <int D>
__device__ __forceinline__ int last_nonfinite(const uint16_t *v, int64_t ts, int first, int end) {
    int found = -1;
    for (int j0 = first; j0 < end; j0 += 64) {
        const int j = j0 + (int)(threadIdx.x & 63);
        uint32_t bad = 0;  // an exponent of ones carries into the bit above
        if (j < end) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                const uint4 w = *reinterpret_cast<const uint4 *>(v + j * ts + 8 * c);
                const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) bad |= (d[e] & 0x7f807f80u) + 0x00800080u;
            }
        }
        const unsigned long long lanes = __ballot((bad & 0x80008000u) != 0);
        if (lanes != 0) found = j0 + 63 - __builtin_clzll(lanes);
    }
    return found;
}

// One query row by a wave from the keys 0..last: 64 keys at a time, a key for each
// lane in the scores, channels for each lane in the weighted sum; a step's keys
// and values are on their way together.
template <int D>
__device__ __forceinline__ void exact_row(const PromptArgs &a, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                                       uint16_t *o, int last) {
    const int lane = threadIdx.x & 63;
    constexpr int kPer = D / 64;
    uint32_t qw = reinterpret_cast<const uint32_t *>(q)[lane % (D / 2)];  // two channels for each lane
    float m = kNegInf, l = 0.0f, acc[kPer] = {};
    auto chunk = [&](int j0, auto whole_c) {
        constexpr bool kWhole = decltype(whole_c)::value;
        const bool mine = kWhole || j0 + lane <= last;
        const uint4 *kr = reinterpret_cast<const uint4 *>(k + (int64_t)(mine ? j0 + lane : last) * a.k_ts);
        uint4 kw[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) kw[c] = kr[c];
        const uint16_t *at = v + (int64_t)j0 * a.v_ts + lane * kPer;
        auto value = [&]() {
            asm("" : "+v"(at));  // one address of the lane's, not 64 of the wave's
            const uint32_t w = kPer == 2 ? *reinterpret_cast<const uint32_t *>(at) : *at;
            at += a.v_ts;
            return w;
        };
        uint32_t vw[kWhole ? 64 : 1];
        if (kWhole) {
#pragma unroll
            for (int i = 0; i < 64; ++i) vw[i] = value();
        }
        float s = 0.0f;
        asm("" : "+v"(qw));  // read out anew in each step, not kept in scalar registers
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            const uint32_t kd[4] = {kw[c].x, kw[c].y, kw[c].z, kw[c].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t qd = (uint32_t)__builtin_amdgcn_readlane((int)qw, 4 * c + e);
                s = fmaf(__uint_as_float(qd << 16), __uint_as_float(kd[e] << 16), s);
                s = fmaf(__uint_as_float(qd & 0xffff0000u), __uint_as_float(kd[e] & 0xffff0000u), s);
            }
        }
        s = mine ? s * a.scale : kNegInf;
        const float m1 = fmaxf(m, wave_max_f(s));
        const float f = m1 == kNegInf ? 1.0f : exp2_fast(m - m1);
        m = m1;
        const float p = mine ? exp2_fast(s - (m == kNegInf ? 0.0f : m)) : 0.0f;
        l = l * f + p;
#pragma unroll
        for (int x = 0; x < kPer; ++x) acc[x] *= f;
        auto add = [&](int i, uint32_t w) {
            const float pi = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(p), i));
            acc[0] = fmaf(pi, __uint_as_float(w << 16), acc[0]);
            if (kPer == 2) acc[kPer - 1] = fmaf(pi, __uint_as_float(w & 0xffff0000u), acc[kPer - 1]);
        };
        if (kWhole) {
#pragma unroll
            for (int i = 0; i < 64; ++i) add(i, vw[kWhole ? i : 0]);
        } else {
#pragma unroll 1
            for (int i = 0; j0 + i <= last; ++i) add(i, value());
        }
    };
    int j0 = 0;
    for (; j0 + 63 <= last; j0 += 64) chunk(j0, std::true_type{});
    if (j0 <= last) chunk(j0, std::false_type{});
    for (int x = 32; x >= 1; x /= 2) l += __shfl_xor(l, x, 64);
    for (int x = 0; x < kPer; ++x) {
        const float r = l != 0.0f ? acc[x] / l : 0.0f;
        o[lane * kPer + x] = (uint16_t)(pack_bf16(r, 0.0f) & 0xffffu);
    }
}

// The rank-th tile of the call: its sequence and its place there.  Workgroups
// start in the order of the ranks, so the tiles with the most keys come first;
// a light tile at the end fills a gap, a heavy one would be waited for.  With a
// causal mask tile i of a sequence counts i + 1 + (prefix in tiles): F(x), the
// number of tiles that count more than x, is summed over the sequences by the
// lanes, and the x with F(x) <= rank < F(x - 1) found by halving.  Without one,
// and beyond 64 sequences, sequence b owns the ranks from q0 / kRows + b on, q0 its
// first row (room for its rows whatever its length), last tiles first.
template <bool CAUSAL, int kRows>
__device__ __forceinline__ bool find_tile(const PromptArgs &a, int rank, int *seq, int *tile, Rows *rows) {
    const int lane = threadIdx.x & 63;
    if (CAUSAL && a.B <= 64) {
        int n = 0, pre = 0, start = lane < a.B ? clamp_row(a.cu_q[lane], a.Tq) : 0;
        if (a.B > 1) start = wave_scan_max(start);
        Rows of = {0, 0};
        if (lane < a.B) {
            of = rows_of(start, a.cu_q[lane + 1], start, a.Tq);
            const int k0 = clamp_row(a.cu_k[lane], a.Tk), nk = max(clamp_row(a.cu_k[lane + 1], a.Tk) - k0, 0);
            n = (of.n + kRows - 1) / kRows, pre = max(nk - of.n, 0) / kRows;
        }
        if (a.B == 1) {
            *seq = 0, *tile = uniform(n) - 1 - rank;
            *rows = Rows{uniform(of.first), uniform(of.n)};
            return *tile >= 0;
        }
        auto above = [&](int x) { return uniform(wave_sum(min(max(n + pre - x, 0), n))); };
        int lo = 0, hi = (a.Tq > a.Tk ? a.Tq : a.Tk) / kRows + 2;  // F(lo) > rank >= F(hi)
        if (above(lo) <= rank) return false;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (above(mid) > rank)
                lo = mid;
            else
                hi = mid;
        }
        // the tiles that count hi: at most one of a sequence
        const bool has = hi > pre && hi <= n + pre;
        const unsigned long long mine = __ballot(has);
        const int skip = rank - above(hi);
        const bool it = has && __popcll(mine & ((1ull << lane) - 1)) == skip;
        *seq = uniform(__builtin_ctzll(__ballot(it)));
        *tile = hi - 1 - uniform(__shfl(pre, *seq, 64));
        *rows = Rows{uniform(__shfl(of.first, *seq, 64)), uniform(__shfl(of.n, *seq, 64))};
        return true;
    }
    const int at = a.tiles - 1 - rank;
    int b = -1, first = 0, floor = 0;
    for (int base = 0; base < a.B; base += 64) {
        const int start =
            max(floor, wave_scan_max(base + lane < a.B ? clamp_row(a.cu_q[min(base + lane, a.B - 1)], a.Tq) : 0));
        const unsigned long long in = __ballot(base + lane < a.B && start / kRows + base + lane <= at);
        if (in == 0) break;
        b = base + __popcll(in) - 1;  // the starts do not fall, so these are the first lanes
        first = __builtin_amdgcn_readlane(start, b - base);
        floor = __builtin_amdgcn_readlane(start, 63);
        if (in != ~0ull) break;
    }
    b = uniform(b);
    if (b < 0) return false;
    *seq = b;
    *tile = at - first / kRows - b;
    *rows = rows_of(first, a.cu_q[b + 1], first, a.Tq);
    return true;
}

// What row r of a V tile is exchanged by.  A transposing read takes 4 rows x 64
// bytes for lanes 0..31 and the 4 rows behind for the others: the rows' 64-byte
// pieces go to different banks, and the two halves to different 32 bytes.
template <int D>
__device__ __forceinline__ int value_place(int r) {
    return (D == 128 ? (r & 3) << 2 : ((r >> 1) & 1) << 2) | (((r >> 2) & 1) << 1);
}

// Whole prompts.  K and V go from memory straight into LDS, in tiles of 64 keys
// that the 4 waves of a workgroup share, one tile ahead; a wave keeps its 32 rows'
// queries and sums in registers.  Two workgroups fit a CU, each with its own
// barrier, so one computes while the other waits.  Bound by the matrix and vector
// instructions together: for 64 rows of a SIMD and a tile 1.2 us of products, 0.7
// of exponentials and the rest; the prompt of 8192 tokens (64 heads of 128
// channels) runs in 1.00 to 1.07 ms by the card, 1030 to 1100 TFLOP/s, where a large
// bf16 product reaches 1305.  With 64 channels half of the products stand beside as many exponentials:
// 890 TFLOP/s.  Measured and left: 256 rows and 8 waves that share a tile (-1 %
// and +1 % on long prompts, +13 % on packed ones), rings of 3 and 4 tiles (one
// workgroup per CU: +20 to +70 %).
//
// A workgroup takes 128 / W query rows of one head, 32 for each of 4 / W pairs
// (W = 2) or single waves (W = 1).  The waves of a pair have the two halves of
// every tile's keys and are joined at the end: twice the workgroups with half of
// the work, for calls with few rows.
//
// SPLIT: a tile's keys are cut once more, into slices of whole tiles of keys for
// workgroups of their own, for a few rows against many keys.  The one that
// finishes last adds the parts in their order (see "Partial results" below).
template <int D, bool CAUSAL, int W, bool SPLIT>
__global__ __launch_bounds__(256, 2) void attn_prompt_kernel(PromptArgs a) {
    static_assert(W == 2 || !SPLIT, "all four waves join, two for 32 rows");
    constexpr int kRows = 128 / W, kBlocks = 2 / W;      // blocks of 32 keys of a wave and tile
    constexpr int kTileBytes = kKeys * D * 2;
    constexpr int kRowBytes = D * 2;
    constexpr int kRowsPerLoad = 1024 / kRowBytes;       // rows that one wave-wide load covers
    constexpr int kLoads = kTileBytes / 1024 / 4;        // loads of one tile per wave
    // Tiles of K and of V in the ring: 64 KB, so that two workgroups fit a CU.
    constexpr int kStages = D == 128 ? 2 : 4;
    __shared__ __attribute__((aligned(1024))) char lds[kStages * 2 * kTileBytes];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), half = lane >> 5, col = lane & 31;
    const int row_wave = wave / W, first_block = W == 1 ? 0 : wave % W;
    if (SPLIT && (int)blockIdx.x == a.tiles * a.Hq - 1 && (int)blockIdx.y == a.slices - 1) clear_next<256>(a.clear);

    // Workgroups go round the 8 XCDs: where the heads divide by 8, each XCD takes
    // the same ones of every tile, so that its L2 holds few heads' keys.
    const int rank = (int)(blockIdx.x / (uint32_t)a.Hq), j = (int)(blockIdx.x - (uint32_t)rank * a.Hq);
    const int head = a.Hq % 8 == 0 ? (j & 7) * (a.Hq / 8) + (j >> 3) : j;
    const int kvh = head / (a.Hq / a.H);
    int b, tile;
    Rows of;
    if (!find_tile<CAUSAL, kRows>(a, rank, &b, &tile, &of)) return;
    const int q0 = of.first, nq = of.n;
    const int k0 = clamp_row(a.cu_k[b], a.Tk), keys = max(clamp_row(a.cu_k[b + 1], a.Tk) - k0, 0);
    const int row0 = tile * kRows;
    if (row0 >= nq) return;

    const int kend = CAUSAL ? min(keys, min(row0 + kRows, nq) + keys - nq) : keys;  // past every row of the workgroup
    int ntiles = kend > 0 ? (kend + kKeys - 1) / kKeys : 0, parts = 1, skip = 0;
    if (SPLIT) {
        const int worth = uniform((int)__builtin_sqrtf(kSliceJoin * (float)ntiles));
        const int per = max(ntiles < kSliceLeast ? ntiles : max((ntiles + a.slices - 1) / a.slices, worth), 1);
        parts = max((ntiles + per - 1) / per, 1);
        if ((int)blockIdx.y >= parts) return;
        const int first = per * (int)blockIdx.y;
        ntiles = min(per, ntiles - first), skip = first * kKeys;
    }
    // from here on keys count from the first of the slice
    const int nk = SPLIT ? min(keys - skip, max(ntiles, 0) * kKeys) : keys, off = keys - skip - nq;
    const int w0 = row0 + 32 * row_wave, row = w0 + col;
    const int last = CAUSAL ? min(nk - 1, row + off) : nk - 1;  // the row's last visible key
    const int wlo = CAUSAL ? min(nk - 1, w0 + off) : nk - 1;    // the same of the wave's first and last row
    const int whi = CAUSAL ? min(nk - 1, min(w0 + 31, nq - 1) + off) : nk - 1;
    const bool live = w0 < nq;

    const uint16_t *qp = a.q + (int64_t)(q0 + min(row, nq - 1)) * a.q_ts + head * a.q_hs;
    const char *kp = reinterpret_cast<const char *>(a.k + (int64_t)(k0 + skip) * a.k_ts + kvh * a.k_hs);
    const char *vp = reinterpret_cast<const char *>(a.v + (int64_t)(k0 + skip) * a.v_ts + kvh * a.v_hs);

    bf8_t qf[D / 16];
#pragma unroll
    for (int t = 0; t < D / 16; ++t) qf[t] = *reinterpret_cast<const bf8_t *>(qp + 16 * t + 8 * half);

    // LDS tiles: row r, 16-byte piece c of it at place c ^ f(r), so that reads
    // down a column of pieces spread over the banks.  A load fills its 1 KB in
    // lane order; the lane picks the piece that belongs there.  Load i of the
    // wave covers rows (4 i + wave) kRowsPerLoad ..., whose f does not depend on i.
    const int lrow = wave * kRowsPerLoad + lane / (kRowBytes / 16), lpiece = lane % (kRowBytes / 16);
    const int fk = D == 128 ? (lrow & 15) : ((lrow >> 1) & 7);
    const int fv = value_place<D>(lrow);
    uint32_t kvo[kLoads], vvo[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        kvo[i] = (uint32_t)((lrow + 4 * kRowsPerLoad * i) * a.k_ts * 2 + (lpiece ^ fk) * 16);
        vvo[i] = (uint32_t)((lrow + 4 * kRowsPerLoad * i) * a.v_ts * 2 + (lpiece ^ fv) * 16);
    }
    const uint32_t lds0 = lds_address(lds + wave * 1024);
    // Past the last tile the loads give zeros, so that every wave has the same
    // number of them on the way.
    auto fetch = [&](const char *base, const uint32_t (&vo)[kLoads], int64_t ts, int t, int which) {
        const int64_t j0 = (int64_t)t * kKeys, left = (nk - 1 - j0) * ts * 2 + kRowBytes;
        const i4_t d = descriptor(base + j0 * ts * 2, t < ntiles ? (uint32_t)min(left, (int64_t)0x7fffffff) : 0);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            load_to_lds(lds0 + (2 * (t % kStages) + which) * kTileBytes + i * 4096, vo[i], d);
    };
    auto fetch_k = [&](int t) { fetch(kp, kvo, a.k_ts, t, 0); };
    auto fetch_v = [&](int t) { fetch(vp, vvo, a.v_ts, t, 1); };

    // reads: K piece 2 t + half of row 32 kb + col; V^T through 4-row blocks
    const int xk = D == 128 ? (col & 15) : ((col >> 1) & 7);
    const uint32_t kbase = col * kRowBytes + ((half ^ (xk & 1)) << 4);
    const int vr = 4 * half + ((lane & 15) >> 2);
    const int xv = value_place<D>(vr);
    const int vsub = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const uint32_t vbase = vr * kRowBytes + ((vsub ^ (xv & 3)) << 4) + (lane & 1) * 8;

    f16_t acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = f16_t{};
    float m = kNegInf, l = 0.0f;

    // scores of 4 of the D / 16 channel steps of a 32-key block
    auto score_step = [&](f16_t &s, const char *kt, int kb, int i) {
        const bf8_t kf = *reinterpret_cast<const bf8_t *>(kt + (first_block + kb) * 32 * kRowBytes + kbase + (((2 * i) ^ (xk & ~1)) << 4));
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[i], s, 0, 0, 0);
    };
    auto scores = [&](f16_t (&s)[kBlocks], int t) {
        const char *kt = lds + (2 * (t % kStages)) * kTileBytes;
#pragma unroll
        for (int kb = 0; kb < kBlocks; ++kb) {
            s[kb] = f16_t{};
#pragma unroll
            for (int i = 0; i < D / 16; ++i) score_step(s[kb], kt, kb, i);
        }
    };
    auto value_step = [&](const char *vt, int u, int i, bf8_t pf) {
        const char *at = vt + (32 * first_block + 16 * u) * kRowBytes + vbase + (((4 * i) ^ (xv & ~3)) << 4);
        const s4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS s4_t *)at);
        const s4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS s4_t *)(at + 8 * kRowBytes));
        const s8_t vv = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8_t, vv), pf, acc[i], 0, 0, 0);
    };

    // Softmax and values of tile t, whose scores are in s, and beside it the
    // scores of tile t + 1 into s: the matrix unit works on one while the
    // vector unit works on the other.
    auto step = [&](f16_t (&s)[kBlocks], int t, auto masked_c, auto next_c) {
        constexpr bool kMasked = decltype(masked_c)::value, kNext = decltype(next_c)::value;
        const char *vt = lds + (2 * (t % kStages) + 1) * kTileBytes, *kt = lds + (2 * ((t + 1) % kStages)) * kTileBytes;
        if (kMasked) {
#pragma unroll
            for (int kb = 0; kb < kBlocks; ++kb)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    s[kb][r] =
                        32 * kb + 8 * (r / 4) + (r & 3) > last - t * kKeys - 32 * first_block - 4 * half ? kNegInf : s[kb][r];
        }
        float top = s[0][0];
#pragma unroll
        for (int i = 1; i < 16 * kBlocks; ++i) top = fmaxf(top, s[i / 16][i % 16]);
        top *= a.scale;
        if (__any(top > m + kSlack)) {
            const float m1 = fmaxf(m, max_halves(top));
            const float f = m1 == kNegInf ? 1.0f : exp2_fast(m - m1);
            m = m1;
            l *= f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) acc[i] *= f;
        }
        const float ms = m == kNegInf ? 0.0f : m;
        bf8_t pf[2 * kBlocks];
        f16_t n[kBlocks];
        auto values = [&](int u) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) value_step(vt, u, i, pf[u]);
        };
#pragma unroll
        for (int u = 0; u < 2 * kBlocks; ++u) {
            uint32_t p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float p0 = exp2_fast(fmaf(s[u / 2][8 * (u & 1) + 2 * e], a.scale, -ms));
                const float p1 = exp2_fast(fmaf(s[u / 2][8 * (u & 1) + 2 * e + 1], a.scale, -ms));
                p[e] = pack_bf16(p0, p1);
                l = add_pair(p[e], l);
            }
            pf[u] = __builtin_bit_cast(bf8_t, i4_t{(int)p[0], (int)p[1], (int)p[2], (int)p[3]});
            if (kNext && u < kBlocks) {
                n[u] = f16_t{};
#pragma unroll
                for (int i = 0; i < D / 16; ++i) score_step(n[u], kt, u, i);
            } else if (u >= kBlocks) {
                values(u - kBlocks);
            }
        }
#pragma unroll
        for (int u = kBlocks; u < 2 * kBlocks; ++u) values(u);
        if (kNext) {
#pragma unroll
            for (int kb = 0; kb < kBlocks; ++kb) s[kb] = n[kb];
        }
    };

    // The keys run one tile ahead of the values: iteration t reads V of tile t
    // and K of t + 1, and sends for V of t + kStages - 1 and K of t + kStages, into
    // the places that iteration t - 1 has read.
    const int mine = live && whi >= 0 ? whi / kKeys + 1 : 0;  // tiles that a row of the wave sees
    f16_t s[kBlocks];
    fetch_k(0);
#pragma unroll
    for (int i = 0; i + 1 < kStages; ++i) {
        fetch_v(i);
        fetch_k(i + 1);
    }
    wait_loads_barrier<(kStages - 1) * 2 * kLoads>();
    // the compiler sees the queries arrive here: it does not know of the loads
    // into LDS, and its waits for the queries inside the loop would wait for those
#pragma unroll
    for (int i = 0; i < D / 16; ++i) asm volatile("" : "+v"(qf[i]));
    if (mine > 0) scores(s, 0);
    auto arrive = [&](int t) {
        wait_loads_barrier<(kStages - 2) * 2 * kLoads>();  // K of t + 1 and V of t are here
        fetch_v(t + kStages - 1);
        fetch_k(t + kStages);
    };
    // tiles that all rows of the wave see whole, then those that hold some row's
    // end, then those that only other waves need
    const int plain = min(mine - 1, (wlo + 1) / kKeys);
    int t = 0;
    for (; t < plain; ++t) {
        arrive(t);
        step(s, t, std::false_type{}, std::true_type{});
    }
    for (; t < mine - 1; ++t) {
        arrive(t);
        step(s, t, std::true_type{}, std::true_type{});
    }
    if (t < mine) {
        arrive(t);
        step(s, t, std::true_type{}, std::false_type{});
        ++t;
    }
    for (; t < ntiles; ++t) arrive(t);
    l = sum_halves(l);
    if (W == 2) {  // the second wave of a pair hands its part to the first
        float *hand = reinterpret_cast<float *>(lds) + row_wave * 32 * (D + 4);
        float *stat = reinterpret_cast<float *>(lds) + 2 * 32 * (D + 4) + row_wave * 64;
        wait_vm0();  // the loads past the last tile, which write zeros
        __syncthreads();
        if (first_block == 1) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int r = 0; r < 16; r += 4)
                    *reinterpret_cast<f4_t *>(hand + col * (D + 4) + 32 * i + 2 * r + 4 * half) =
                        f4_t{acc[i][r], acc[i][r + 1], acc[i][r + 2], acc[i][r + 3]};
            if (half == 0) stat[col] = m, stat[32 + col] = l;
        }
        __syncthreads();
    }
    auto redo_rows = [&](uint32_t todo) {  // of the wave's rows, those with a bit, where hidden values may be why
        if (!CAUSAL || todo == 0) return;
        const uint16_t *values = a.v + (int64_t)k0 * a.v_ts + kvh * a.v_hs;
        auto last_of = [&](int r) { return min(keys - 1, r + keys - nq); };
        // past the keys of the wave's last tile
        const int past = min(keys, (max(last_of(min(w0 + 31, nq - 1)), -1) / kKeys + 1) * kKeys);
        const int hidden = last_nonfinite<D>(values, a.v_ts, max(last_of(w0), -1) + 1, past);
        for (; todo != 0; todo &= todo - 1) {
            const int r = w0 + __builtin_ctz(todo), last_key = last_of(r);
            if (last_key >= hidden) continue;
            exact_row<D>(a, a.q + (int64_t)(q0 + r) * a.q_ts + head * a.q_hs, a.k + (int64_t)k0 * a.k_ts + kvh * a.k_hs,
                         values, a.o + ((int64_t)(q0 + r) * a.Hq + head) * D, last_key);
        }
    };
    if (W == 2 && first_block == 0) {
        const float *hand = reinterpret_cast<const float *>(lds) + row_wave * 32 * (D + 4);
        const float *stat = reinterpret_cast<const float *>(lds) + 2 * 32 * (D + 4) + row_wave * 64;
        const float m2 = stat[col], l2 = stat[32 + col], m1 = fmaxf(m, m2);
        const float f1 = m == kNegInf ? 0.0f : exp2_fast(m - m1), f2 = m2 == kNegInf ? 0.0f : exp2_fast(m2 - m1);
        m = m1, l = l * f1 + l2 * f2;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const f4_t o = *reinterpret_cast<const f4_t *>(hand + col * (D + 4) + 32 * i + 2 * r + 4 * half);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][r + e] = acc[i][r + e] * f1 + o[e] * f2;
            }
    }
    uint16_t *op = a.o + ((int64_t)(q0 + row) * a.Hq + head) * D;
    if (SPLIT && parts > 1) {
        __shared__ int arrived;
        __shared__ uint32_t bad_rows[4];
        constexpr int kSlot = kRows * (D + 2), kPart = D / 8;  // pairs of sums that a lane joins
        const float *parts0 = a.part + (int64_t)blockIdx.x * a.slices * kSlot;
        if (live && first_block == 0) {
            float *at = a.part + ((int64_t)blockIdx.x * a.slices + blockIdx.y) * kSlot;
            if (half == 0) store_agent(at + 2 * (32 * row_wave + col), m, l);
            at += 2 * kRows + row_wave * 32 * D + 2 * lane;
#pragma unroll
            for (int i = 0; i < D / 4; ++i) store_agent(at + i * 128, acc[i / 8][2 * (i % 8)], acc[i / 8][2 * (i % 8) + 1]);
        }
        wait_vm0();
        __syncthreads();
        if (tid == 0)
            arrived = __hip_atomic_fetch_add(a.counts + blockIdx.x, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (uniform(arrived) != parts - 1) return;
        // each wave of a pair joins half of the channels, the next part's reads under way
        uint32_t todo = 0;
        if (live) {
            float2 ml, next_ml, part[kPart], next[kPart], sum[kPart];
            auto read = [&](int g) {
                const float *p = parts0 + (int64_t)g * kSlot;
                next_ml = load_agent(p + 2 * (32 * row_wave + col));
                p += 2 * kRows + row_wave * 32 * D + 2 * lane + first_block * kPart * 128;
#pragma unroll
                for (int i = 0; i < kPart; ++i) next[i] = load_agent(p + i * 128);
            };
            m = kNegInf, l = 0.0f;
#pragma unroll
            for (int i = 0; i < kPart; ++i) sum[i] = make_float2(0.0f, 0.0f);
            read(0);
#pragma unroll 1
            for (int g = 0; g < parts; ++g) {
                ml = next_ml;
#pragma unroll
                for (int i = 0; i < kPart; ++i) part[i] = next[i];
                if (g + 1 < parts) read(g + 1);
                const float m1 = fmaxf(m, ml.x);
                const float f0 = m == kNegInf ? 0.0f : exp2_fast(m - m1), f1 = ml.x == kNegInf ? 0.0f : exp2_fast(ml.x - m1);
                m = m1, l = l * f0 + ml.y * f1;
#pragma unroll
                for (int i = 0; i < kPart; ++i)
                    sum[i] = make_float2(sum[i].x * f0 + part[i].x * f1, sum[i].y * f0 + part[i].y * f1);
            }
            const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
            bool bad = false;
#pragma unroll
            for (int e = 0; e < kPart; e += 2) {
                const float x[4] = {sum[e].x * inv, sum[e].y * inv, sum[e + 1].x * inv, sum[e + 1].y * inv};
#pragma unroll
                for (int c = 0; c < 4; ++c) bad |= !(fabsf(x[c]) < __builtin_huge_valf());
                if (row < nq)
                    *reinterpret_cast<uint2 *>(op + first_block * (D / 2) + 32 * (e / 8) + 4 * (e % 8) + 4 * half) =
                        make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
            }
            const unsigned long long redo = __ballot(bad && row < nq);
            todo = (uint32_t)(redo | redo >> 32);
        }
        if (tid == 0) __hip_atomic_store(a.counts + blockIdx.x, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (lane == 0) bad_rows[wave] = todo;
        wait_vm0();  // a row that is redone is written after both of its halves
        __syncthreads();
        if (first_block == 0) redo_rows(uniform((int)(bad_rows[wave] | bad_rows[wave + 1])));
        return;
    }
    if (!live || first_block == 1) return;
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);  // l NaN stays NaN
    bool bad = false;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = acc[i][r + e] * inv;
                bad |= !(fabsf(x[e]) < __builtin_huge_valf());
            }
            if (row < nq)
                *reinterpret_cast<uint2 *>(op + 32 * i + 2 * r + 4 * half) =
                    make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
        }
    unsigned long long redo = __ballot(bad && row < nq);
    redo_rows((uint32_t)(redo | redo >> 32));
}

// ================================================================== cache ==
struct CacheArgs {
    const uint16_t *q;
    const uint8_t *codes;
    const float *scales;
    const int32_t *table, *lens, *cu_q;  // cu_q null: one row per sequence
    const uint64_t *tree;                // null: causal
    uint16_t *o;
    float *part;   // partial results
    int *counts;   // workgroups that have finished with an item, by the first of them
    int *clear;    // the next call's counters
    int64_t q_ts, q_hs, max_pages, pages;
    int B, Tq, Hq, H, G, page_shift, groups;
    float scale;
};

// What a sequence asks for: its rows, and the units of its items (qw3_units.h).
// All items of the call, laid end to end, are cut into equal runs of units, one
// per workgroup (fewer workgroups where the runs would be too short for their
// join): a long sequence is split over many workgroups and short ones share one,
// with no lengths known on the host.
template <int R>
struct Seq {
    int q0, nq, len, blocks, per_item, units;
    __device__ Seq() {}
    __device__ Seq(const CacheArgs &a, int b, int floor) {  // floor: the largest start before (without cu_q: any)
        const Rows rows = a.cu_q ? rows_of(a.cu_q[b], a.cu_q[b + 1], floor, a.Tq) : Rows{b, 1};
        q0 = rows.first, nq = rows.n;
        len = a.pages == 0 ? 0 : (int)max((int64_t)0, min((int64_t)a.lens[b], a.max_pages << a.page_shift));
        blocks = blocks_of(nq * a.G, R);
        per_item = units_of_item(len, R);
        units = per_item * blocks * a.H;
    }
};

// What adding one workgroup's part costs in the join, in units.  A run of u units
// leaves an item of n units in n / u parts that one workgroup adds, u + kJoin n / u
// in all, least at u = sqrt(kJoin n): runs are no shorter than that for the longest
// item.  Without it a long sequence of few heads is cut for the whole card and
// waits for its join.  Measured without, and with 0.07, 0.14, 0.8: one kv head, one
// token over 30000 keys 32, 18, 17 and 25 us, over 131071 46, 32, 31, 48; with rows
// of 128 or 256 without, and with 0.1, 0.5, 0.8, 1.0: trees of 64 over 6000 keys of
// one kv head 193, 88, 62, 57, 71 us.  Short items lose 0.1 us to the root.
template <int R>
constexpr float kJoin = R <= 32 ? 0.14f : 0.8f;

// A workgroup's run of units: [u, end) of the call's total, beginning in
// sequence b, before which there are `before` units and whose starts' floor is `floor`.
struct Work {
    int per, u, end, before, b, floor;
};
template <int R>
__device__ __forceinline__ Work find_work(const CacheArgs &a) {
    const int lane = threadIdx.x & 63;
    int total = 0, mine = 0, upto = 0, longest = 0, floor = 0, start = 0;
    // the lane's sequence of 64: its units, and the largest start up to its own
    auto sequence = [&](int b) {
        if (a.cu_q) start = max(floor, wave_scan_max(b < a.B ? clamp_row(a.cu_q[min(b, a.B)], a.Tq) : 0));
        mine = 0;
        if (b < a.B) {
            const Seq<R> seq(a, b, start);
            mine = seq.units;
            if (mine > 0) longest = max(longest, seq.per_item);
        }
    };
    for (int base = 0; base < a.B; base += 64) {
        sequence(base + lane);
        upto = total + wave_scan(mine);
        total = __builtin_amdgcn_readlane(upto, 63);
        if (a.B > 64) floor = __builtin_amdgcn_readlane(start, 63);
    }
    const int least = uniform((int)__builtin_sqrtf(kJoin<R> * (float)wave_max(longest)));
    const Run run = run_of(total, a.groups, least, blockIdx.x);
    Work work = {run.per, run.begin, run.end, 0, 0, 0};
    if (work.u >= work.end || a.B == 1) return work;
    int done = 0;
    floor = 0;
    for (int base = 0; base < a.B; base += 64) {
        if (a.B > 64) {
            sequence(base + lane);
            upto = done + wave_scan(mine);
        }
        const unsigned long long past = __ballot(upto > work.u);
        if (past) {
            const int at = uniform(__builtin_ctzll(past));
            work.b = base + at;
            work.before = __builtin_amdgcn_readlane(upto - mine, at);
            work.floor = __builtin_amdgcn_readlane(start, at);
            break;
        }
        done = __builtin_amdgcn_readlane(upto, 63);
        floor = __builtin_amdgcn_readlane(start, 63);
    }
    return work;
}

// Partial results.  An item that several workgroups worked on is joined by the
// one that finishes last.  A slot holds R maxima, R sums and R x D weighted
// sums; a workgroup has two, for its first and its last item (those between are
// its own).  Slots are written and read by atomic 8-byte accesses of agent
// scope, which go past the per-XCD L2s, so no cache has to be flushed; every
// thread's stores are complete (vmcnt 0) before its workgroup counts itself.
// The count belongs to the first workgroup of the item; the joining workgroup sets
// it back to zero, and the call clears the bank that the next one counts in.
template <int R, int D>
__device__ __forceinline__ float *partial(const CacheArgs &a, int group, int which) {
    return a.part + (int64_t)(group * 2 + which) * (R * (D + 2));
}
// NaN among e4m3 codes.  A place that was never written may hold one, and a weight
// of zero does not hide it (0 NaN = NaN).  So where a tile has keys that some row
// may not see, the codes that are NaN go to the matrix unit as zeros, and NaN goes
// into just the sums of the rows that see them: what a row does not see has no
// influence on it, and one that sees a NaN has it in that channel.

// The bytes of w that are NaN (0x7f, 0xff), each with its highest bit.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t without_codes(uint32_t w, uint32_t n) { return w & ~(n | (n - (n >> 7))); }
__device__ __forceinline__ uint4 nan_codes(uint4 w) {
    return make_uint4(nan_codes(w.x), nan_codes(w.y), nan_codes(w.z), nan_codes(w.w));
}
__device__ __forceinline__ uint4 without_codes(uint4 w, uint4 n) {
    return make_uint4(without_codes(w.x, n.x), without_codes(w.y, n.y), without_codes(w.z, n.z), without_codes(w.w, n.w));
}
__device__ __forceinline__ uint32_t any_of(uint4 n) { return n.x | n.y | n.z | n.w; }
constexpr float kNaN = __builtin_nanf("");

// The keys base..base + 63 that a row sees, as bits: all up to `seen`, and of
// the drafts, which begin at ctx, those of its word; none from len on.
__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1; }
__device__ __forceinline__ uint64_t visible(int base, int seen, uint64_t tree, int ctx, int len) {
    const int at = ctx - base;
    const uint64_t drafts = at >= 64 || at <= -64 ? 0 : at >= 0 ? tree << at : tree >> -at;
    return (low_bits(seen + 1 - base) | drafts) & low_bits(len - base);
}

// Few rows: R = 16 or 32 query rows of an item.  Every wave takes all R rows
// and 32 of the unit's keys; codes and scales go from memory to registers a
// step ahead, K's straight as the matrix unit's operand, V's through a tile of
// the wave's own in LDS that turns them.  The waves meet only at the end of an
// item.  Bound by memory where there is much of it (64 sequences of 2048 tokens
// 56 us, 4.9 TB/s, what a large copy reaches; one of 131071 tokens 61 us, of
// which 8 join 62 parts a head), and by its own chain of dependent reads where
// there is little: one token over 1000 keys 8.5 us in a graph, of which 1.1 find
// the work, 0.8 a page number, 1.1 the codes, 1.6 the step with its instructions,
// 1.2 join the waves, 2.6 the parts.  Three workgroups a CU (168 registers,
// spills) measured 73 us where two measure 56; codes by direct loads into LDS,
// with the compiler's waits for all of them, 104 us where 61 are measured now.
template <int D, bool E4M3, int R>
__global__ __launch_bounds__(256, 2) void attn_few_kernel(CacheArgs a) {
    constexpr int kUnit = unit_of(R);
    constexpr int kN = R / 16;                   // blocks of 16 rows
    constexpr int kCols = R == 16 ? D : 64;      // channels joined at a time
    constexpr int kPad = kCols + 4;
    constexpr int kTurn = 4 * 32 * D, kJoin = 4 * R * kPad * 4;
    __shared__ __attribute__((aligned(1024))) char lds[kTurn > kJoin ? kTurn : kJoin];
    __shared__ float stat[2][4][R];
    __shared__ int arrived[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), quarter = lane >> 4, col = lane & 15;

    Work run = find_work<R>(a);
    if ((int)blockIdx.x == a.groups - 1) clear_next<R <= 32 ? 256 : 2 * R>(a.clear);  // it has work in large calls only
    if (run.u >= run.end) return;
    Seq<R> seq(a, run.b, run.floor);

    constexpr int kPieces = D / 16, kVLoads = D / 32;
    // V tile: row r, 16-byte piece c at place c ^ f(r), so that the turning reads spread over the banks
    char *turn = lds + wave * 32 * D;
    auto place = [](int r) { return D == 128 ? (r >> 1) & 7 : (r >> 2) & 3; };
    const int vrow = lane / kPieces, vpiece = lane % kPieces;

    struct Stage {
        uint4 k[2][D / 64], v[kVLoads];
        float4 ks[2], vs[2];
    };

    // the portion of an item that is worked on: units t0.. of it, for the rows
    // r0.. of kv head h of a sequence, the wave's keys 32 from key0 + 128 s in step s
    int h, r0, rows, q0, len, ctx, key0, steps;
    int ustart, count;  // the item's first unit; units of the portion
    const int32_t *table;
    auto locate = [&]() {
        while (run.u - run.before >= seq.units) {  // next sequence (some have no rows)
            run.before += seq.units;
            if (++run.b >= a.B) return false;  // only if the arrays change under the call
            seq = Seq<R>(a, run.b, seq.q0 + seq.nq);
        }
        const int item = (int)((uint32_t)(run.u - run.before) / (uint32_t)seq.per_item);
        const int begin = run.before + item * seq.per_item;
        ustart = begin + kSetup;
        run.u = max(run.u, ustart);
        const int t0 = run.u - ustart;
        count = min(begin + seq.per_item, run.end) - run.u;
        if (count <= 0) return false;  // the run ends before the item's first keys
        h = (int)((uint32_t)item / (uint32_t)seq.blocks);
        r0 = (item - h * seq.blocks) * R;
        rows = seq.nq * a.G, q0 = seq.q0, len = seq.len, ctx = len - seq.nq;
        key0 = t0 * kUnit + 32 * wave;
        steps = len <= key0 ? 0 : min(count, (len - key0 + kUnit - 1) / kUnit);
        table = a.table + (int64_t)run.b * a.max_pages;
        return true;
    };
    if (!locate()) return;

        // pages of 32 steps: lane 2 s + g has the one of group g (16 keys) of step s
        auto pages_of = [&](int s) {
            const int pos = min(key0 + (s + (lane >> 1)) * kUnit + 16 * (lane & 1), len - 1);
            return table[pos >> a.page_shift];
        };
        int ids = 0, ids_next = 0, ids_base = 0;
        auto begin_ids = [&]() {
            ids_base = 0;
            if (steps > 0) ids = pages_of(0);
            if (steps > 32) ids_next = pages_of(32);
        };
        const int64_t page_rows = (int64_t)(2 * a.H) << a.page_shift;
        const int64_t to_v = (int64_t)a.H << a.page_shift;
        auto page_of = [&](int s, int g) { return __builtin_amdgcn_readlane(ids, 2 * (s - ids_base) + g); };
        Stage st;
        auto fetch = [&](int s) {
            const int key = key0 + s * kUnit;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                // a group past the end reads the last key's, a page that does not exist page 0: hidden below
                const int pos = min(key + 16 * g, (len - 1) & ~15);
                int page = page_of(s, g);
                page = (uint32_t)page < (uint64_t)a.pages ? page : 0;
                const int64_t row = page * page_rows + ((int64_t)h << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
                const uint8_t *kp = a.codes + row * D, *vp = kp + to_v * D;
                const float *sp = a.scales + row;
                // a uniform base and a lane's offset: kept apart, or the compiler makes
                // a 64-bit address for each lane and load
                uint32_t ko = col * D + quarter * 16, vo = lane * 16, so = 4 * quarter;
                asm("" : "+v"(ko), "+v"(vo), "+v"(so));
#pragma unroll
                for (int c = 0; c < D / 64; ++c) st.k[g][c] = *reinterpret_cast<const uint4 *>(kp + ko + 64 * c);
#pragma unroll
                for (int c = 0; c < kVLoads / 2; ++c)
                    st.v[g * (kVLoads / 2) + c] = *reinterpret_cast<const uint4 *>(vp + vo + 1024 * c);
                st.ks[g] = *reinterpret_cast<const float4 *>(sp + so);
                st.vs[g] = *reinterpret_cast<const float4 *>(sp + to_v + so);
            }
        };

        // the rows' queries, as B operands with the channels in the order of K's pieces
        bf8_t qf[kN][D / 32];
        int seen[kN];       // causal: the row's last visible key
        uint64_t tree[kN];  // otherwise the drafts it sees
        auto begin_loads = [&]() {
            if (steps > 0) fetch(0);
#pragma unroll
            for (int x = 0; x < kN; ++x) {
                const int r = min(r0 + 16 * x + col, rows - 1), i = r / a.G, g = r - i * a.G;
                const uint16_t *qp = a.q + (int64_t)(q0 + i) * a.q_ts + (h * a.G + g) * a.q_hs;
#pragma unroll
                for (int t = 0; t < D / 32; ++t)
                    qf[x][t] = *reinterpret_cast<const bf8_t *>(qp + 16 * (quarter + 4 * (t / 2)) + 8 * (t & 1));
                seen[x] = a.tree ? ctx - 1 : ctx + i;
                tree[x] = a.tree ? a.tree[q0 + i] : 0;
            }
        };
        begin_ids();
        begin_loads();

        f4_t acc[kN][D / 16];
        float m[kN], l[kN];

        auto step = [&](int s, auto masked_c) {
            constexpr bool kMasked = decltype(masked_c)::value;
            const int key = key0 + s * kUnit;
            bool gone[2] = {false, false};
            if (kMasked) {
#pragma unroll
                for (int g = 0; g < 2; ++g) gone[g] = (uint32_t)page_of(s, g) >= (uint64_t)a.pages;
            }
            // V's codes into the turning tile
            uint32_t nans_here = 0;
#pragma unroll
            for (int c = 0; c < kVLoads; ++c) {
                const int r = vrow + c * (64 / kPieces);
                if (E4M3 && kMasked) {
                    if (key + r >= len || gone[c / (kVLoads / 2)]) st.v[c] = make_uint4(0, 0, 0, 0);
                    nans_here |= nan_codes(st.v[c].x) | nan_codes(st.v[c].y) | nan_codes(st.v[c].z) | nan_codes(st.v[c].w);
                }
                *reinterpret_cast<uint4 *>(turn + r * D + ((vpiece ^ place(r)) << 4)) = st.v[c];
            }
            if (E4M3 && kMasked && __any(nans_here != 0)) {
                uint32_t nan_keys = 0;  // of the wave's 32, as bits
#pragma unroll
                for (int c = 0; c < kVLoads; ++c) {
                    const int r = vrow + c * (64 / kPieces);
                    const uint4 w = st.v[c], nans = nan_codes(w);
                    *reinterpret_cast<uint4 *>(turn + r * D + ((vpiece ^ place(r)) << 4)) = without_codes(w, nans);
                    for (unsigned long long lanes = __ballot(any_of(nans) != 0); lanes != 0;) {
                        const int row = __builtin_ctzll(lanes) / kPieces;
                        nan_keys |= 1u << (row + c * (64 / kPieces));
                        lanes &= ~(((1ull << kPieces) - 1) << (row * kPieces));
                    }
                }
                for (; nan_keys != 0; nan_keys &= nan_keys - 1) {
                    const int r = __builtin_ctz(nan_keys);  // its page exists, or its codes were taken as zeros
                    const int64_t row = page_of(s, r >> 4) * page_rows + ((int64_t)h << a.page_shift) + to_v +
                                        ((key + r) & ((1 << a.page_shift) - 1));
                    const uint8_t *at = a.codes + row * D + 4 * quarter;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const uint32_t nans = nan_codes(*reinterpret_cast<const uint32_t *>(at + 16 * i));
#pragma unroll
                        for (int x = 0; x < kN; ++x)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if ((nans >> (8 * e + 7)) & (uint32_t)(visible(key, seen[x], tree[x], ctx, len) >> r) & 1)
                                    acc[x][i][e] = kNaN;
                    }
                }
            }
            float kc[2][4], vc[2][4];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                kc[g][0] = st.ks[g].x * a.scale, kc[g][1] = st.ks[g].y * a.scale;
                kc[g][2] = st.ks[g].z * a.scale, kc[g][3] = st.ks[g].w * a.scale;
                vc[g][0] = st.vs[g].x, vc[g][1] = st.vs[g].y, vc[g][2] = st.vs[g].z, vc[g][3] = st.vs[g].w;
                // copies, so that the next step's loads land in the same registers and
                // are not waited for at the end of this one
#pragma unroll
                for (int r = 0; r < 4; ++r) asm volatile("" : "+v"(vc[g][r]));
            }
            f4_t sc[kN][2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
#pragma unroll
                for (int x = 0; x < kN; ++x) sc[x][g] = f4_t{};
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const uint4 w = st.k[g][c];
                    const bf8_t k0 = decode8<E4M3>(w.x, w.y), k1 = decode8<E4M3>(w.z, w.w);
#pragma unroll
                    for (int x = 0; x < kN; ++x) {
                        sc[x][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, qf[x][2 * c], sc[x][g], 0, 0, 0);
                        sc[x][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, qf[x][2 * c + 1], sc[x][g], 0, 0, 0);
                    }
                }
            }
            if (!kMasked || s + 1 < steps) {
                if (s + 1 == ids_base + 32) {
                    ids = ids_next, ids_base += 32;
                    if (ids_base + 32 < steps) ids_next = pages_of(ids_base + 32);
                }
                fetch(s + 1);
            }
            // A weight is the sum of two bf16: its rounding and the rounding of what that
            // leaves (16 bits).  One would do for a flat softmax; where one key decides a
            // row, its error is that of every channel.  The second costs 8 of 24 matrix
            // instructions of a kernel that waits for memory.
            bf8_t pf[kN], pl[kN];
#pragma unroll
            for (int x = 0; x < kN; ++x) {
                bool hid[2][4];
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        sc[x][g][r] *= kc[g][r];
                        hid[g][r] = false;
                    }
                if (kMasked) {
                    uint64_t vis = visible(key, seen[x], tree[x], ctx, len);
                    if (gone[0]) vis &= ~0xffffull;
                    if (gone[1]) vis &= ~0xffff0000ull;
                    vis >>= 4 * quarter;
#pragma unroll
                    for (int g = 0; g < 2; ++g)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            hid[g][r] = !((vis >> (16 * g + r)) & 1);
                            sc[x][g][r] = hid[g][r] ? kNegInf : sc[x][g][r];
                        }
                }
                float top = sc[x][0][0];
#pragma unroll
                for (int i = 1; i < 8; ++i) top = fmaxf(top, sc[x][i / 4][i % 4]);
                if (__any(top > m[x] + kSlack)) {
                    const float m1 = fmaxf(m[x], max_quarters(top));
                    const float f = m1 == kNegInf ? 1.0f : exp2_fast(m[x] - m1);
                    m[x] = m1;
                    l[x] *= f;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) acc[x][i] *= f;
                }
                const float ms = m[x] == kNegInf ? 0.0f : m[x];
                uint32_t p[4], pr[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float w[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int g = i / 2, r = 2 * (i & 1) + e;
                        const float pe = exp2_fast(sc[x][g][r] - ms);
                        l[x] += pe;
                        // a hidden key's scale may be anything
                        w[e] = kMasked && hid[g][r] ? 0.0f : pe * vc[g][r];
                    }
                    p[i] = pack_bf16(w[0], w[1]);
                    pr[i] = pack_bf16(w[0] - __uint_as_float(p[i] << 16), w[1] - __uint_as_float(p[i] & 0xffff0000u));
                }
                pf[x] = __builtin_bit_cast(bf8_t, i4_t{(int)p[0], (int)p[1], (int)p[2], (int)p[3]});
                pl[x] = __builtin_bit_cast(bf8_t, i4_t{(int)pr[0], (int)pr[1], (int)pr[2], (int)pr[3]});
            }
            // V^T: keys 4 quarter + 0..3 and 16 + 4 quarter + 0..3 of 16 channels
            const int vkey = 4 * quarter + ((col >> 1) & 3) + 16 * (col >> 3), xv = place(vkey);
            const char *from = turn + vkey * D + (col & 1) * 8;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const i2_t w = __builtin_amdgcn_ds_read_tr8_b64_v2i32((LDS_AS i2_t *)(from + ((i ^ xv) << 4)));
                const bf8_t vf = decode8<E4M3>((uint32_t)w[0], (uint32_t)w[1]);
#pragma unroll
                for (int x = 0; x < kN; ++x) {
                    acc[x][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[x], acc[x][i], 0, 0, 0);
                    acc[x][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pl[x], acc[x][i], 0, 0, 0);
                }
            }
        };
    // items shared with other workgroups (at most the first and the last)
    struct Shared {
        int first, last, slot, h, r0, n, q0;  // slot: where the first workgroup's part is
    } shared[2];
    int nshared = 0;
    for (;;) {
#pragma unroll
        for (int x = 0; x < kN; ++x) {
            m[x] = kNegInf, l[x] = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) acc[x][i] = f4_t{};
        }
        // steps up to the first that can hold a draft, the end or a missing page, then the others
        const int plain = min(steps - 1, (min(ctx, len) - key0 - 32 + kUnit) / kUnit);
        int s = 0;
        for (; s < plain; ++s) {
            if ((uint32_t)page_of(s, 0) >= (uint64_t)a.pages || (uint32_t)page_of(s, 1) >= (uint64_t)a.pages) break;
            step(s, std::false_type{});
        }
        for (; s < steps; ++s) step(s, std::true_type{});

        // the next portion's page numbers and then its first loads are on their way
        // while this one's waves are joined
        const int first = group_of(ustart, run.per);
        const Shared done = {first, group_of(ustart + seq.per_item - kSetup - 1, run.per),
                             first * run.per == ustart ? 0 : 1, h, r0, min(R, rows - r0), q0};
        float *out = nullptr;
        if (done.first != done.last) {
            out = partial<R, D>(a, blockIdx.x, first < (int)blockIdx.x || first * run.per == ustart ? 0 : 1);
            if (nshared == 0)
                shared[0] = done;
            else
                shared[1] = done;
            ++nshared;
        }
        run.u += count;
        const bool more = run.u < run.end && locate();
        if (more) begin_ids();
#pragma unroll
        for (int x = 0; x < kN; ++x) {
            l[x] = sum_quarters(l[x]);
            if (quarter == 0) stat[0][wave][16 * x + col] = m[x], stat[1][wave][16 * x + col] = l[x];
        }
        float *join = reinterpret_cast<float *>(lds);
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += kCols) {
            lds_barrier();  // the turning tiles, or the channels before, are read
#pragma unroll
            for (int x = 0; x < kN; ++x)
#pragma unroll
                for (int i = 0; i < kCols / 16; ++i)
                    *reinterpret_cast<f4_t *>(join + (wave * R + 16 * x + col) * kPad + 16 * i + 4 * quarter) =
                        acc[x][c0 / 16 + i];
            if (more && c0 + kCols == D) begin_loads();
            lds_barrier();
            for (int e = tid; e < done.n * kCols / 2; e += 256) {
                const int r = e / (kCols / 2), c = 2 * (e % (kCols / 2));
                float mm = kNegInf;
#pragma unroll
                for (int w = 0; w < 4; ++w) mm = fmaxf(mm, stat[0][w][r]);
                float ll = 0.0f;
                f2_t sum = {};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float f = stat[0][w][r] == kNegInf ? 0.0f : exp2_fast(stat[0][w][r] - mm);
                    ll += f * stat[1][w][r];
                    sum += f * *reinterpret_cast<const f2_t *>(join + (w * R + r) * kPad + c);
                }
                if (out == nullptr) {
                    const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
                    const int i = (done.r0 + r) / a.G, g = done.r0 + r - i * a.G;
                    *reinterpret_cast<uint32_t *>(a.o + ((int64_t)(done.q0 + i) * a.Hq + done.h * a.G + g) * D + c0 + c) =
                        pack_bf16(sum[0] * inv, sum[1] * inv);
                } else {
                    store_agent(out + 2 * R + r * D + c0 + c, sum[0], sum[1]);
                    if (c0 == 0 && c == 0) store_agent(out + 2 * r, mm, ll);
                }
            }
        }
        lds_barrier();
        if (!more) break;
    }

    if (nshared == 0) return;
    wait_vm0();
    __syncthreads();
    if (tid < nshared)
        arrived[tid] = __hip_atomic_fetch_add(a.counts + (tid == 0 ? shared[0].first : shared[1].first), 1,
                                              __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < nshared; ++i) {
        const Shared s = i == 0 ? shared[0] : shared[1];
        if (uniform(arrived[i]) != s.last - s.first) continue;
        const float *from = partial<R, D>(a, s.first, s.slot);
        auto slot_of = [&](int g) -> const float * { return g == s.first ? from : partial<R, D>(a, g, 0); };
        auto row_out = [&](int r) {
            const int i = (s.r0 + r) / a.G, g = s.r0 + r - i * a.G;
            return a.o + ((int64_t)(s.q0 + i) * a.Hq + s.h * a.G + g) * D;
        };
        if (s.n <= R / 2)
            join_rows<R, D, R / 8>(slot_of, s.first, s.last, s.n, row_out);
        else
            join_rows<R, D, R / 4>(slot_of, s.first, s.last, s.n, row_out);
        if (tid == 0) __hip_atomic_store(a.counts + s.first, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

// Many rows: R = 128 or 256 query rows of an item, 32 for each wave; the waves
// share tiles of 64 keys.  The tile's codes come through registers a tile ahead
// and are turned into bf16 once for all waves; the rest is attn_prompt_kernel's.
// Bound by matrix and vector instructions: the two scales of a key and the
// conversion make about 430 vector instructions beside 32 products (1.2 of the
// 1.4 us that a tile takes a wave), 770 TFLOP/s on long caches, and 25 us of a
// call are the exchange of partial results (trees of 64 drafts over 36,000
// tokens, 512 rows a kv head: 130 us).  256 rows halve the conversion: 129 us
// where 128 rows take 134.
template <int D, bool E4M3, int R>
__global__ __launch_bounds__(2 * R, 2) void attn_many_kernel(CacheArgs a) {
    constexpr int kUnit = unit_of(R);             // 64
    constexpr int kThreads = 2 * R;               // a wave for each 32 rows
    static_assert(kUnit * (D / 16) % kThreads == 0, "every thread has the same pieces of a tile");
    constexpr int kRowBytes = D * 2, kTileBytes = kUnit * kRowBytes;
    constexpr int kPieces = D / 16;               // 16-byte pieces of a row of codes
    constexpr int kLoads = kUnit * kPieces / kThreads;  // of a thread, for K and for V
    __shared__ __attribute__((aligned(1024))) char lds[4 * kTileBytes];  // K, V of two tiles
    __shared__ __attribute__((aligned(16))) float tile_scales[2][2][kUnit];
    __shared__ uint32_t tile_nans[E4M3 ? 2 : 1][kUnit];  // keys with values that are NaN
    __shared__ int arrived[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), half = lane >> 5, col = lane & 31;

    Work run = find_work<R>(a);
    if ((int)blockIdx.x == a.groups - 1) clear_next<R <= 32 ? 256 : 2 * R>(a.clear);  // it has work in large calls only
    if (run.u >= run.end) return;
    Seq<R> seq(a, run.b, run.floor);

    const int lrow = tid / kPieces, lpiece = tid % kPieces;  // of a thread's first load; the others kThreads / kPieces rows on
    const int xk = D == 128 ? (col & 15) : ((col >> 1) & 7);
    const uint32_t kbase = col * kRowBytes + ((half ^ (xk & 1)) << 4);
    const int vr = 4 * half + ((lane & 15) >> 2), xv = value_place<D>(vr);
    const int vsub = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const uint32_t vbase = vr * kRowBytes + ((vsub ^ (xv & 3)) << 4) + (lane & 1) * 8;

    struct Shared {
        int first, last, slot, h, r0, n, q0;  // slot: where the first workgroup's part is
    } shared[2];
    int nshared = 0;
    while (run.u < run.end) {
        while (run.u - run.before >= seq.units) {  // next sequence (some have no rows)
            run.before += seq.units;
            if (++run.b >= a.B) break;  // only if the arrays change under the call
            seq = Seq<R>(a, run.b, seq.q0 + seq.nq);
        }
        if (run.b >= a.B) break;
        const int item = (int)((uint32_t)(run.u - run.before) / (uint32_t)seq.per_item);
        const int begin = run.before + item * seq.per_item, ustart = begin + kSetup;
        run.u = max(run.u, ustart);
        const int t0 = run.u - ustart, count = min(begin + seq.per_item, run.end) - run.u;
        if (count <= 0) break;  // the run ends before the item's first keys
        const int h = (int)((uint32_t)item / (uint32_t)seq.blocks), r0 = (item - h * seq.blocks) * R;
        const int rows = seq.nq * a.G, q0 = seq.q0, len = seq.len, ctx = len - seq.nq;
        const int key0 = t0 * kUnit;
        const int tiles = min(count, (len - key0 + kUnit - 1) / kUnit);
        const int32_t *table = a.table + (int64_t)run.b * a.max_pages;

        // page numbers of 16 tiles: lane 4 t + g has the one of 16-key group g of tile t
        int ids = 0, ids_next = 0, ids_base = 0;
        auto pages_of = [&](int t) {
            return table[min(key0 + (t + (lane >> 2)) * kUnit + 16 * (lane & 3), len - 1) >> a.page_shift];
        };
        if (tiles > 0) ids = pages_of(0);
        if (tiles > 16) ids_next = pages_of(16);
        const int64_t page_rows = (int64_t)(2 * a.H) << a.page_shift, to_v = (int64_t)a.H << a.page_shift;
        const int in_page = (1 << a.page_shift) - 1;
        auto row_of = [&](int t, int r) {  // row of the codes of key r of tile t; its page exists, or it is hidden
            int page = __shfl(ids, 4 * (t - ids_base) + (r >> 4), 64);
            page = (uint32_t)page < (uint64_t)a.pages ? page : 0;
            return page * page_rows + ((int64_t)h << a.page_shift) + (min(key0 + t * kUnit + r, len - 1) & in_page);
        };
        uint4 kcode[kLoads], vcode[kLoads];
        float scale_in = 0.0f;
        uint32_t gone_in = 0;  // groups of the tile whose page does not exist
        auto fetch = [&](int t) {
            if (t == ids_base + 16) {
                ids = ids_next, ids_base += 16;
                if (ids_base + 16 < tiles) ids_next = pages_of(ids_base + 16);
            }
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const uint8_t *at = a.codes + row_of(t, lrow + i * (kThreads / kPieces)) * D + lpiece * 16;
                kcode[i] = *reinterpret_cast<const uint4 *>(at);
                vcode[i] = *reinterpret_cast<const uint4 *>(at + to_v * D);
            }
            const int64_t srow = row_of(t, tid & 63);
            if (tid < 128) scale_in = a.scales[srow + (tid < 64 ? 0 : to_v)];
            const unsigned long long missing = __ballot((uint32_t)ids >= (uint64_t)a.pages);
            gone_in = uniform((int)((missing >> (4 * (t - ids_base))) & 15));
        };
        uint32_t gone = 0;  // of the tile in LDS
        auto partly = [&](int t) { return key0 + (t + 1) * kUnit > min(ctx, len) || gone_in != 0; };  // of the fetched tile
        bool mixed = false;  // the tile in LDS has keys that some row may not see
        auto place = [&](int t) {  // the fetched tile, as bf16, into its buffer
            char *kt = lds + (2 * (t & 1)) * kTileBytes, *vt = kt + kTileBytes;
            const bool clean = E4M3 && partly(t);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int r = lrow + i * (kThreads / kPieces);
                const int fk = D == 128 ? (r & 15) : ((r >> 1) & 7), fv = value_place<D>(r);
                *reinterpret_cast<bf8_t *>(kt + r * kRowBytes + (((2 * lpiece) ^ fk) << 4)) =
                    decode8<E4M3>(kcode[i].x, kcode[i].y);
                *reinterpret_cast<bf8_t *>(kt + r * kRowBytes + (((2 * lpiece + 1) ^ fk) << 4)) =
                    decode8<E4M3>(kcode[i].z, kcode[i].w);
                uint4 w = vcode[i], nans = make_uint4(0, 0, 0, 0);
                if (clean) {
                    if (key0 + t * kUnit + r >= len || ((gone_in >> (r >> 4)) & 1)) w = make_uint4(0, 0, 0, 0);
                    nans = nan_codes(w);
                    w = without_codes(w, nans);
                    const unsigned long long lanes = __ballot(any_of(nans) != 0);
                    if (lpiece == 0) tile_nans[t & 1][r] = (uint32_t)(lanes >> lane) & ((1u << kPieces) - 1);
                }
                bf8_t v0 = decode8<E4M3>(w.x, w.y), v1 = decode8<E4M3>(w.z, w.w);
                if (clean && __any(any_of(nans) != 0)) {
                    // in the tile such a value is 2^-133, which no code stands for
                    auto mark = [](bf8_t v, uint32_t lo, uint32_t hi) {
                        i4_t x = __builtin_bit_cast(i4_t, v);
                        x[0] |= (int)((lo >> 7 & 1) | (lo >> 15 & 1) << 16), x[1] |= (int)((lo >> 23 & 1) | (lo >> 31 & 1) << 16);
                        x[2] |= (int)((hi >> 7 & 1) | (hi >> 15 & 1) << 16), x[3] |= (int)((hi >> 23 & 1) | (hi >> 31 & 1) << 16);
                        return __builtin_bit_cast(bf8_t, x);
                    };
                    v0 = mark(v0, nans.x, nans.y), v1 = mark(v1, nans.z, nans.w);
                }
                *reinterpret_cast<bf8_t *>(vt + r * kRowBytes + (((2 * lpiece) ^ fv) << 4)) = v0;
                *reinterpret_cast<bf8_t *>(vt + r * kRowBytes + (((2 * lpiece + 1) ^ fv) << 4)) = v1;
            }
            if (tid < 128) tile_scales[t & 1][tid >> 6][tid & 63] = tid < 64 ? scale_in * a.scale : scale_in;
        };

        // the lane's query row
        const int row = min(r0 + 32 * wave + col, rows - 1), tok = row / a.G;
        const bool live = r0 + 32 * wave < rows;
        const uint16_t *qp = a.q + (int64_t)(q0 + tok) * a.q_ts + (h * a.G + row - tok * a.G) * a.q_hs;
        bf8_t qf[D / 16];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) qf[i] = *reinterpret_cast<const bf8_t *>(qp + 16 * i + 8 * half);
        const int seen = a.tree ? ctx - 1 : ctx + tok;
        const uint64_t tree = a.tree ? a.tree[q0 + tok] : 0;

        f16_t acc[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) acc[i] = f16_t{};
        float m = kNegInf, l = 0.0f;

        auto step = [&](int t, auto masked_c) {
            constexpr bool kMasked = decltype(masked_c)::value;
            const char *kt = lds + (2 * (t & 1)) * kTileBytes, *vt = kt + kTileBytes;
            f16_t s[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                s[b] = f16_t{};
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const bf8_t kf =
                        *reinterpret_cast<const bf8_t *>(kt + b * 32 * kRowBytes + kbase + (((2 * i) ^ (xk & ~1)) << 4));
                    s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[i], s[b], 0, 0, 0);
                }
            }
            uint64_t vis = 0;  // of the keys that the lane has, from bit 0 on
            if (kMasked) {
                vis = visible(key0 + t * kUnit, seen, tree, ctx, len);
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    if ((gone >> g) & 1) vis &= ~(0xffffull << (16 * g));
                if (E4M3 && mixed) {
                    for (unsigned long long left = __ballot(tile_nans[t & 1][lane] != 0); left != 0; left &= left - 1) {
                        const int r = uniform(__builtin_ctzll(left));
                        const char *at = vt + r * kRowBytes + 8 * half;
#pragma unroll
                        for (int i = 0; i < D / 32; ++i)
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                const s4_t v = *reinterpret_cast<const s4_t *>(at + (((4 * i + e / 4) ^ value_place<D>(r)) << 4));
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    if (v[c] == 1 && ((vis >> r) & 1)) acc[i][e + c] = kNaN;
                            }
                    }
                }
                vis >>= 4 * half;
            }
            float top = kNegInf;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const f4_t ks = *reinterpret_cast<const f4_t *>(&tile_scales[t & 1][0][32 * b + 2 * r + 4 * half]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = s[b][r + e] * ks[e];
                        if (kMasked && !((vis >> (32 * b + 2 * r + e)) & 1)) x = kNegInf;
                        s[b][r + e] = x;
                        top = fmaxf(top, x);
                    }
                }
            }
            if (__any(top > m + kSlack)) {
                const float m1 = fmaxf(m, max_halves(top));
                const float f = m1 == kNegInf ? 1.0f : exp2_fast(m - m1);
                m = m1;
                l *= f;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) acc[i] *= f;
            }
            const float ms = m == kNegInf ? 0.0f : m;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t p[4];
#pragma unroll
                    for (int r = 0; r < 8; r += 4) {
                        const f4_t vs = *reinterpret_cast<const f4_t *>(
                            &tile_scales[t & 1][1][32 * b + 2 * (8 * u + r) + 4 * half]);
                        float w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = s[b][8 * u + r + e], pe = exp2_fast(x - ms);
                            l += pe;
                            // a hidden key's scale may be anything
                            w[e] = kMasked && x == kNegInf ? 0.0f : pe * vs[e];
                        }
                        p[r / 2] = pack_bf16(w[0], w[1]), p[r / 2 + 1] = pack_bf16(w[2], w[3]);
                    }
                    const bf8_t pf = __builtin_bit_cast(bf8_t, i4_t{(int)p[0], (int)p[1], (int)p[2], (int)p[3]});
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        const char *at = vt + (32 * b + 16 * u) * kRowBytes + vbase + (((4 * i) ^ (xv & ~3)) << 4);
                        const s4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS s4_t *)at);
                        const s4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS s4_t *)(at + 8 * kRowBytes));
                        const s8_t vv = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                        acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8_t, vv), pf, acc[i], 0, 0, 0);
                    }
                }
            }
        };

        if (tiles > 0) {
            fetch(0);
            place(0);
            gone = gone_in, mixed = partly(0);
        }
        auto iteration = [&](int t, auto masked_c) {
            lds_barrier();  // tile t is in place; nobody reads the other buffer any more
            if (t + 1 < tiles) fetch(t + 1);
            if (live) step(t, masked_c);
            if (t + 1 < tiles) {
                place(t + 1);
                gone = gone_in, mixed = partly(t + 1);
            }
        };
        // tiles up to the first that can hold a draft, the end or a missing page, then the others
        const int plain = min(tiles, (min(ctx, len) - key0) / kUnit);
        int t = 0;
        for (; t < plain && gone == 0; ++t) iteration(t, std::false_type{});
        for (; t < tiles; ++t) iteration(t, std::true_type{});

        const int first = group_of(ustart, run.per), last = group_of(begin + seq.per_item - 1, run.per);
        float *out = nullptr;
        if (first != last) {
            out = partial<R, D>(a, blockIdx.x, first < (int)blockIdx.x || first * run.per == ustart ? 0 : 1);
            const Shared mine = {first, last, first * run.per == ustart ? 0 : 1, h, r0, min(R, rows - r0), q0};
            if (nshared == 0)
                shared[0] = mine;
            else
                shared[1] = mine;
            ++nshared;
        }
        l = sum_halves(l);
        lds_barrier();  // the last tile is read
        const int r = 32 * wave + col;  // of the item
        if (r0 + r < rows) {
            if (out == nullptr) {
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                uint16_t *op = a.o + ((int64_t)(q0 + tok) * a.Hq + h * a.G + row - tok * a.G) * D;
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<uint2 *>(op + 32 * i + 2 * e + 4 * half) =
                            make_uint2(pack_bf16(acc[i][e] * inv, acc[i][e + 1] * inv),
                                       pack_bf16(acc[i][e + 2] * inv, acc[i][e + 3] * inv));
            } else {
                // in the order of the registers, so that a wave's stores are contiguous
                float *at = out + 2 * R + wave * 32 * D + 2 * lane;
#pragma unroll
                for (int i = 0; i < D / 4; ++i)
                    store_agent(at + i * 128, acc[i / 8][2 * (i % 8)], acc[i / 8][2 * (i % 8) + 1]);
                if (half == 0) store_agent(out + 2 * r, m, l);
            }
        }
        run.u += count;
    }

    if (nshared == 0) return;
    wait_vm0();
    __syncthreads();
    if (tid < nshared)
        arrived[tid] = __hip_atomic_fetch_add(a.counts + (tid == 0 ? shared[0].first : shared[1].first), 1,
                                              __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < nshared; ++i) {
        const Shared s = i == 0 ? shared[0] : shared[1];
        if (uniform(arrived[i]) != s.last - s.first) continue;
        const int r = 32 * wave + col;
        if (32 * wave < s.n) {
            // a lane joins what it and its like have stored, in the workgroups' order; the
            // reads of the next part are under way while one is added
            auto slot = [&](int g) { return partial<R, D>(a, g, g == s.first ? s.slot : 0); };
            float2 ml, next_ml, part[D / 4], next[D / 4];
            auto read = [&](int g) {
                const float *p = slot(g), *at = p + 2 * R + wave * 32 * D + 2 * lane;
                next_ml = load_agent(p + 2 * min(r, s.n - 1));
#pragma unroll
                for (int i = 0; i < D / 4; ++i) next[i] = load_agent(at + i * 128);
            };
            float m = kNegInf, l = 0.0f;
            float2 sum[D / 4];
#pragma unroll
            for (int i = 0; i < D / 4; ++i) sum[i] = make_float2(0.0f, 0.0f);
            read(s.first);
#pragma unroll 1
            for (int g = s.first; g <= s.last; ++g) {
                ml = next_ml;
#pragma unroll
                for (int i = 0; i < D / 4; ++i) part[i] = next[i];
                if (g < s.last) read(g + 1);
                const float m1 = fmaxf(m, ml.x);
                const float f0 = m == kNegInf ? 0.0f : exp2_fast(m - m1), f1 = ml.x == kNegInf ? 0.0f : exp2_fast(ml.x - m1);
                m = m1, l = l * f0 + ml.y * f1;
#pragma unroll
                for (int i = 0; i < D / 4; ++i)
                    sum[i] = make_float2(sum[i].x * f0 + part[i].x * f1, sum[i].y * f0 + part[i].y * f1);
            }
            if (r < s.n) {
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                const int i = (s.r0 + r) / a.G, g = s.r0 + r - i * a.G;
                uint16_t *op = a.o + ((int64_t)(s.q0 + i) * a.Hq + s.h * a.G + g) * D;
#pragma unroll
                for (int e = 0; e < D / 4; e += 2)
                    *reinterpret_cast<uint2 *>(op + 32 * (e / 8) + 4 * (e % 8) + 4 * half) =
                        make_uint2(pack_bf16(sum[e].x * inv, sum[e].y * inv),
                                   pack_bf16(sum[e + 1].x * inv, sum[e + 1].y * inv));
            }
        }
        if (tid == 0) __hip_atomic_store(a.counts + s.first, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

bool units_fit(const CacheArgs &a, int R) {
    return qw3_units::units_fit(a.Tq, a.G, a.B, a.H, a.max_pages << a.page_shift, R);
}

template <int D, bool E4M3, int R>
qw3_status launch_cache(CacheArgs a, hipStream_t stream) {
    if (!units_fit(a, R)) return QW3_ERR_SHAPE;
    int cus = 0;
    qw3_status st = cu_count(&cus);
    if (st != QW3_OK) return st;
    a.groups = cus * (R == 256 ? 1 : 2);
    Scratch ws;
    st = workspace(stream, (size_t)a.groups * 2 * R * (D + 2) * sizeof(float), &ws);
    if (st != QW3_OK) return st;
    a.part = static_cast<float *>(ws.ptr);
    st = counters(stream, a.groups, &a.counts, &a.clear);
    if (st != QW3_OK) return st;
    if constexpr (R <= 32)
        hipLaunchKernelGGL((attn_few_kernel<D, E4M3, R>), dim3(a.groups), dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((attn_many_kernel<D, E4M3, R>), dim3(a.groups), dim3(2 * R), 0, stream, a);
    return check_launch();
}

template <int D, bool E4M3>
qw3_status launch_cache_rows(const CacheArgs &a, hipStream_t stream) {
    // Rows of a sequence, on average.  16 drafts of 4 heads a kv head, 64 rows: 55
    // us in blocks of 32, 54 in one of 64 with shared tiles; 52 rows of 64 channels
    // 18 and 31 us.
    const int64_t rows = ceil_div(a.Tq, a.B) * a.G;
    if (rows <= 16) return launch_cache<D, E4M3, 16>(a, stream);
    if (rows <= 64) return launch_cache<D, E4M3, 32>(a, stream);
    // Larger blocks read a key for more rows, smaller ones spread over more
    // workgroups and have less to join.  The host knows the work only by the keys
    // that the table can name.  Trees of 64, 512 rows a kv head of 128 channels, in
    // blocks of 32, 128 and 256: 1 kv head over 1500 keys 17, 26 and 36 us, over 6000
    // 30, 42, 57; 4 sequences of 8 over 1500 keys 39, 43, 54, over 6000 117, 88, 86; 8
    // sequences of 8 over 1500..8000 214, 132, 129.  With 64 channels in blocks of 32
    // and 128: 2 kv heads over 6000 keys 24 and 29 us, 8 39 and 35.
    if (a.Tq * (int64_t)a.Hq * (a.max_pages << a.page_shift) <= (D == 128 ? 1 << 25 : 1 << 24))
        return launch_cache<D, E4M3, 32>(a, stream);
    if (!units_fit(a, 128)) return QW3_ERR_SHAPE;  // before the device is asked: no device decides on a refusal
    int cus = 0;
    const qw3_status st = cu_count(&cus);
    if (st != QW3_OK) return st;
    if (D == 128 && rows > 128 && (int64_t)a.Tq * a.Hq >= int64_t(256) * (cus / 2))  // blocks of 256 for half of the CUs
        return launch_cache<D, E4M3, D == 128 ? 256 : 128>(a, stream);
    return launch_cache<D, E4M3, 128>(a, stream);
}

// Row strides: 64 rows' offsets stay in a buffer descriptor's 31 bits.
bool strides_ok(int64_t ts, int64_t hs) { return qw3_shared::strides_ok(ts, hs, 1 << 23); }

qw3_status check_heads(int64_t Hq, int64_t H) {
    return H < 1 || Hq < 1 || Hq % H != 0 || Hq > QW3_MAX_HEADS ? QW3_ERR_SHAPE : QW3_OK;
}

bool scale_ok(float s) { return s > 0.0f && s < __builtin_huge_valf(); }

}  // namespace

// Four banks per (device, stream handle), cleared by the first call on the stream
// and never grown: kCounts is more than any grid that counts.
namespace {
struct Counters {
    int dev;
    hipStream_t stream;
    int *ptr;
    Banks banks;
};
std::mutex g_counters_mutex;
std::vector<Counters> g_counters;
__global__ void clear_counts_kernel(int *p) { p[blockIdx.x * 256 + threadIdx.x] = 0; }

qw3_status clear_counts(int *p, int banks, hipStream_t stream) {
    hipLaunchKernelGGL(clear_counts_kernel, dim3(banks * kCounts / 256), dim3(256), 0, stream, p);
    return check_launch();
}
}  // namespace

qw3_status qw3_shared::counters(hipStream_t stream, int n, int **use, int **clear) {
    if (n > kCounts) return hip_fail(hipErrorInvalidValue);
    int dev = 0;
    hipError_t err = hipGetDevice(&dev);
    if (err != hipSuccess) return hip_fail(err);
    hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
    unsigned long long id = 0;
    if (hipStreamGetCaptureInfo(stream, &capture, &id) != hipSuccess) {
        (void)hipGetLastError();
        capture = hipStreamCaptureStatusNone;
    }
    const bool capturing = capture != hipStreamCaptureStatusNone;
    std::lock_guard<std::mutex> lock(g_counters_mutex);
    Counters *mine = nullptr;
    for (auto &e : g_counters)
        if (e.dev == dev && e.stream == stream) mine = &e;
    if (mine == nullptr) {
        if (capturing) return QW3_ERR_CAPTURE;
        if (!qw3_host::room_for_one(g_counters)) return hip_fail(hipErrorOutOfMemory);
        void *p = nullptr;
        err = hipMalloc(&p, 4 * kCounts * sizeof(int));
        if (err != hipSuccess) return hip_fail(err);
        const qw3_status st = clear_counts(static_cast<int *>(p), 4, stream);
        if (st != QW3_OK) {
            (void)hipFree(p);
            return st;
        }
        g_counters.push_back(Counters{dev, stream, static_cast<int *>(p), Banks{}});
        mine = &g_counters.back();
    }
    const BankChoice choice = mine->banks.choose(capturing, id);
    *use = mine->ptr + choice.use * kCounts, *clear = mine->ptr + choice.clear * kCounts;
    return choice.fresh ? clear_counts(mine->ptr + 2 * kCounts, 2, stream) : QW3_OK;
}

extern "C" {

qw3_status qattn_prompt(const uint16_t *q, const uint16_t *k, const uint16_t *v, const int32_t *cu_q,
                        const int32_t *cu_k, uint16_t *out, int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t H,
                        int64_t D, int64_t q_ts, int64_t q_hs, int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs,
                        int32_t causal, float sm_scale, void *hip_stream) {
    if (check_heads(Hq, H) != QW3_OK || (D != 64 && D != 128)) return QW3_ERR_SHAPE;
    if (B < 0 || B > QW3_MAX_SEQS || Tq < 0 || Tk < 0 || Tq > QW3_MAX_TOKENS || Tk > QW3_MAX_TOKENS)
        return QW3_ERR_SHAPE;
    if (!scale_ok(sm_scale) || !strides_ok(q_ts, q_hs) || !strides_ok(k_ts, k_hs) || !strides_ok(v_ts, v_hs))
        return QW3_ERR_SHAPE;
    if ((Tq / 128 + B) * Hq >= kMaxGroups) return QW3_ERR_SHAPE;
    if (B == 0 || Tq == 0) return QW3_OK;
    if (!q || !cu_q || !cu_k || !out || (Tk > 0 && (!k || !v))) return QW3_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(cu_q, 4) ||
        !aligned(cu_k, 4) || q_ts % 8 || q_hs % 8 || k_ts % 8 || k_hs % 8 || v_ts % 8 || v_hs % 8)
        return QW3_ERR_ALIGN;
    PromptArgs a{};
    a.q = q, a.k = k, a.v = v, a.o = out, a.cu_q = cu_q, a.cu_k = cu_k, a.q_ts = q_ts, a.q_hs = q_hs;
    a.k_ts = k_ts, a.k_hs = k_hs, a.v_ts = v_ts, a.v_hs = v_hs, a.B = (int)B, a.Tq = (int)Tq, a.Tk = (int)Tk;
    a.Hq = (int)Hq, a.H = (int)H, a.scale = sm_scale * 1.44269504088896341f;
    int cus = 0;
    qw3_status st = cu_count(&cus);
    if (st != QW3_OK) return st;
    // room for every sequence's last, partly filled tile
    // Halves of 64 rows while 128-row tiles leave CUs with less than two workgroups:
    // measured at 288 tiles (64 channels, 6511 keys) 85 us whole, 79 halved; at 136
    // (4000 tokens, 8 heads) 72 and 55; at 1040 (3..2500 tokens, 16 heads) 63 and 75.
    const bool few = (Tq / 128 + B) * Hq <= 2 * (int64_t)cus;
    const int64_t tiles = Tq / (few ? 64 : 128) + B;
    a.tiles = (int)tiles;
    const hipStream_t stream = (hipStream_t)hip_stream;
    // in slices while the tiles leave half of the CUs' places empty
    a.slices = few && Tk > (kSliceLeast - 1) * kKeys ? (int)std::max<int64_t>(2 * cus / (tiles * Hq), 1) : 1;
    Scratch ws;
    if (a.slices > 1) {
        st = workspace(stream, (size_t)(tiles * Hq * a.slices) * 64 * (D + 2) * sizeof(float), &ws);
        if (st != QW3_OK) return st;
        a.part = static_cast<float *>(ws.ptr);
        st = counters(stream, (int)(tiles * Hq), &a.counts, &a.clear);
        if (st != QW3_OK) return st;
    }
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles * Hq), (unsigned)a.slices), dim3(256), 0, stream, a);
    };
    auto by_mask = [&](auto d, auto w, auto split) {
        constexpr int kD = decltype(d)::value, kW = decltype(w)::value;
        constexpr bool kSplit = decltype(split)::value;
        causal ? run(attn_prompt_kernel<kD, true, kW, kSplit>) : run(attn_prompt_kernel<kD, false, kW, kSplit>);
    };
    auto by_rows = [&](auto d) {
        using One = std::integral_constant<int, 1>;
        using Two = std::integral_constant<int, 2>;
        a.slices > 1 ? by_mask(d, Two{}, std::true_type{})
        : few        ? by_mask(d, Two{}, std::false_type{})
                     : by_mask(d, One{}, std::false_type{});
    };
    D == 128 ? by_rows(std::integral_constant<int, 128>{}) : by_rows(std::integral_constant<int, 64>{});
    return check_launch();
}

qw3_status qattn_cache(const uint16_t *q, const void *codes, const float *scales, int32_t code_type,
                       const int32_t *block_table, const int32_t *lens, const int32_t *cu_q, const int64_t *tree,
                       uint16_t *out, int64_t B, int64_t max_pages, int64_t Tq, int64_t Hq, int64_t H, int64_t D,
                       int64_t pages, int64_t page_size, int64_t q_ts, int64_t q_hs, float sm_scale,
                       void *hip_stream) {
    int shift = 0;
    qw3_status st = check_cache(code_type, H, D, pages, page_size, &shift);
    if (st != QW3_OK) return st;
    if (check_heads(Hq, H) != QW3_OK) return QW3_ERR_SHAPE;
    if (B < 0 || B > QW3_MAX_SEQS || Tq < 0 || Tq > QW3_MAX_TOKENS || max_pages < 0 || (!cu_q && Tq != B))
        return QW3_ERR_SHAPE;
    if (max_pages > (int64_t(1) << 30) / page_size || Tq * Hq > (int64_t(1) << 30)) return QW3_ERR_SHAPE;
    if (!scale_ok(sm_scale) || !strides_ok(q_ts, q_hs)) return QW3_ERR_SHAPE;
    if (B == 0 || Tq == 0) return QW3_OK;
    if (!q || !lens || !out || (max_pages > 0 && !block_table) || (pages > 0 && (!codes || !scales)))
        return QW3_ERR_NULL;
    if (!aligned(q, 16) || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(out, 16) ||
        !aligned(block_table, 4) || !aligned(lens, 4) || !aligned(cu_q, 4) || !aligned(tree, 8) || q_ts % 8 || q_hs % 8)
        return QW3_ERR_ALIGN;
    CacheArgs a{};
    a.q = q, a.codes = static_cast<const uint8_t *>(codes), a.scales = scales, a.table = block_table, a.lens = lens;
    a.cu_q = cu_q, a.tree = reinterpret_cast<const uint64_t *>(tree), a.o = out, a.q_ts = q_ts, a.q_hs = q_hs;
    a.max_pages = max_pages, a.pages = pages, a.B = (int)B, a.Tq = (int)Tq, a.Hq = (int)Hq, a.H = (int)H;
    a.G = (int)(Hq / H), a.page_shift = shift, a.scale = sm_scale * 1.44269504088896341f;
    const hipStream_t stream = (hipStream_t)hip_stream;
    if (D == 128)
        return code_type == QW3_CODES_E4M3 ? launch_cache_rows<128, true>(a, stream)
                                           : launch_cache_rows<128, false>(a, stream);
    return code_type == QW3_CODES_E4M3 ? launch_cache_rows<64, true>(a, stream)
                                       : launch_cache_rows<64, false>(a, stream);
}

}  // extern "C"
