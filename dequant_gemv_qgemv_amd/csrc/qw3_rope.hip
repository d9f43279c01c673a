// Rotary positions on the way from a layer's q/k/v product to its attention:
// qrope rotates rows, qrope_write does it for q and k and writes k and v into the
// quantised cache in the same pass.  C ABI in include/qw3.h.
//
// Pair i < R / 2 of a token's rows is turned by t = p[axis[i]] rates[i] radians, p the
// token's position on each axis: (x, y) -> (x cos t - y sin t, y cos t + x sin t).
// In halves x and y are channels i and i + R / 2, in pairs 2 i and 2 i + 1.
//
// Angles.  Positions go far (2^31) and rates are up to 1 and more, so t is formed
// in 64 bits as turns, t / 2 pi, whose whole part drops out exactly; what is left
// (below half a turn) keeps 24 bits for the sine and cosine in fp32.  All heads of
// a token share its angles: a workgroup computes those of its tokens once, into
// LDS, one angle for each thread.
//
// Bound by memory: each row is read once and written once.  8191 tokens of 64 + 2 x 8
// heads of 128 channels, fp32, three axes, into the cache and dense: 111 us for 336 MB read
// and 186 MB written, 4.7 TB/s; 4081 patches of 32 heads of 64 channels, bf16: 6.5 us, 5.1
// TB/s; 32 tokens of a decode step: 3.9 us.
#include "qw3_quant.h"

using namespace qw3_shared;

namespace {

struct RopeArgs {
    const void *q, *k, *v;
    const int32_t *positions;  // [A, T]
    const double *rates;       // [half]
    const int32_t *axis;       // [half] or null
    const int64_t *slots;
    uint16_t *q_out, *k_out, *v_out;  // k_out and v_out may be null
    uint8_t *codes;
    float *scales;
    int T, Hq, H, half, A;
    int tokens, rows;  // of a workgroup: its tokens, and how many of each token's rows
    int page_shift;
    int64_t n_slots, q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;
};

constexpr int kMostTokens = 4;  // of a workgroup

// A row is taken by D / 16 lanes, 16 channels each, in pieces of 16 bytes of the
// source.  The first R / 16 lanes have the rotated ones, piece m of the first half
// and the same piece of the second, so that a pair's channels meet in one lane and
// the lanes' pieces lie side by side in memory; the others have the rest.  A row
// that goes into the cache is quantised where it is.
template <int D, bool F32, bool E4M3, bool PAIRS, bool CACHE>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a) {
    constexpr int kLanes = D / 16, kRows = 256 / kLanes;
    constexpr int P = F32 ? 4 : 8, kPieces = 16 / P;  // channels of a piece, pieces of a lane
    __shared__ __attribute__((aligned(16))) float2 turns[kMostTokens * D / 2];
    const int tid = threadIdx.x, half = a.half;
    const int t0 = (int)blockIdx.x * a.tokens, nt = min(a.tokens, a.T - t0);
    for (int i = tid; i < nt * half; i += 256) {
        const int t = (int)((uint32_t)i / (uint32_t)half), pair = i - t * half;
        const int ax = a.axis ? min(max(a.axis[pair], 0), a.A - 1) : 0;
        const double x = (double)a.positions[(int64_t)ax * a.T + t0 + t] * (a.rates[pair] * 0.15915494309189533577);
        float s, c;
        sincospif(2.0f * (float)(x - rint(x)), &s, &c);
        turns[i] = make_float2(c, s);
    }
    __syncthreads();

    const int c = tid % kLanes, turned = half / 8;  // lanes that rotate
    const bool rotates = c < turned;
    int off[kPieces];
#pragma unroll
    for (int m = 0; m < kPieces; ++m)
        off[m] = rotates ? P * (c + turned * (m % (kPieces / 2))) + (m >= kPieces / 2 ? half : 0)
                         : 2 * half + P * (c - turned + (kLanes - turned) * m);

    const int all = CACHE ? a.Hq + 2 * a.H : a.Hq;
    const int first = (int)blockIdx.y * a.rows, n = min(a.rows, all - first);
    int t = 0, j = tid / kLanes;
    while (j >= n && t < nt) j -= n, ++t;
    // every lane of a row takes the same branches, so the row's exchanges stay whole
    while (t < nt) {
        const int row = first + j, token = t0 + t;
        const int kind = !CACHE || row < a.Hq ? 0 : row < a.Hq + a.H ? 1 : 2;
        const int h = kind == 0 ? row : kind == 1 ? row - a.Hq : row - a.Hq - a.H;
        const void *src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
        const int64_t at = token * (kind == 0 ? a.q_ts : kind == 1 ? a.k_ts : a.v_ts) +
                           h * (kind == 0 ? a.q_hs : kind == 1 ? a.k_hs : a.v_hs);
        float x[16];
#pragma unroll
        for (int m = 0; m < kPieces; ++m) {
            const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const char *>(src) + (at + off[m]) * (F32 ? 4 : 2));
            const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (F32) {
                    x[4 * m + e] = __uint_as_float(d[e]);
                } else {
                    x[P * m + 2 * e] = __uint_as_float(d[e] << 16);
                    x[P * m + 2 * e + 1] = __uint_as_float(d[e] & 0xffff0000u);
                }
            }
        }
        if (kind < 2 && rotates) {
            const float2 *mine = turns + t * half;
            if (PAIRS) {
#pragma unroll
                for (int m = 0; m < kPieces; ++m)
#pragma unroll
                    for (int e = 0; e < P; e += 2) {
                        const float2 cs = mine[(off[m] + e) / 2];
                        const float u = x[P * m + e], v = x[P * m + e + 1];
                        x[P * m + e] = u * cs.x - v * cs.y;
                        x[P * m + e + 1] = v * cs.x + u * cs.y;
                    }
            } else {
#pragma unroll
                for (int m = 0; m < kPieces / 2; ++m)
#pragma unroll
                    for (int e = 0; e < P; ++e) {
                        const float2 cs = mine[off[m] + e];
                        const float u = x[P * m + e], v = x[P * (m + kPieces / 2) + e];
                        x[P * m + e] = u * cs.x - v * cs.y;
                        x[P * (m + kPieces / 2) + e] = v * cs.x + u * cs.y;
                    }
            }
        }
        uint16_t *dense = kind == 0 ? a.q_out : kind == 1 ? a.k_out : a.v_out;
        if (kind == 0 || dense != nullptr) {
            dense += ((int64_t)token * (kind == 0 ? a.Hq : a.H) + h) * D;
#pragma unroll
            for (int m = 0; m < kPieces; ++m) {
                uint32_t w[P / 2];
#pragma unroll
                for (int e = 0; e < P / 2; ++e) w[e] = pack_bf16(x[P * m + 2 * e], x[P * m + 2 * e + 1]);
                if constexpr (P == 8)
                    *reinterpret_cast<uint4 *>(dense + off[m]) = make_uint4(w[0], w[1], w[2], w[3]);
                else
                    *reinterpret_cast<uint2 *>(dense + off[m]) = make_uint2(w[0], w[1]);
            }
        }
        if (CACHE && kind > 0) {
            const int64_t slot = a.slots[token];
            if (slot >= 0 && slot < a.n_slots) {
                const int64_t page = slot >> a.page_shift;
                const int64_t to = (((page * 2 + kind - 1) * a.H + h) << a.page_shift) + (slot - (page << a.page_shift));
                uint32_t w[4];
                const float s = quantise<D, E4M3>(x, w);
#pragma unroll
                for (int m = 0; m < kPieces; ++m) {
                    uint32_t *dst = reinterpret_cast<uint32_t *>(a.codes + to * D + off[m]);
                    if constexpr (P == 8)
                        *reinterpret_cast<uint2 *>(dst) = make_uint2(w[2 * m], w[2 * m + 1]);
                    else
                        *dst = w[m];
                }
                if (c == 0) a.scales[to] = s;
            }
        }
        j += kRows;
        while (j >= n && t < nt) j -= n, ++t;
    }
}

template <bool CACHE>
qw3_status launch_rope(RopeArgs a, int32_t src_type, int32_t code_type, int64_t D, int32_t style, hipStream_t stream) {
    const int64_t all = CACHE ? a.Hq + 2 * (int64_t)a.H : a.Hq, at_once = 256 / (D / 16);
    // Tokens share a workgroup where there are many; where there are few, one token's
    // rows are spread over several.
    a.tokens = (int64_t)a.T * all >= 16384 ? kMostTokens : 1;
    a.rows = (int)(a.tokens > 1 ? all : at_once);
    const dim3 grid((unsigned)ceil_div(a.T, a.tokens), (unsigned)ceil_div(all, a.rows));
    auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, a); };
    auto by_style = [&](auto d, auto f32, auto e4m3) {
        constexpr int kD = decltype(d)::value;
        constexpr bool kF32 = decltype(f32)::value, kE4M3 = decltype(e4m3)::value;
        style == QW3_ROPE_PAIRS ? run(rope_kernel<kD, kF32, kE4M3, true, CACHE>)
                                : run(rope_kernel<kD, kF32, kE4M3, false, CACHE>);
    };
    auto by_type = [&](auto d, auto f32) {
        if constexpr (CACHE) {
            code_type == QW3_CODES_E4M3 ? by_style(d, f32, std::true_type{}) : by_style(d, f32, std::false_type{});
        } else {
            by_style(d, f32, std::false_type{});
        }
    };
    auto by_source = [&](auto d) {
        src_type == QW3_SRC_F32 ? by_type(d, std::true_type{}) : by_type(d, std::false_type{});
    };
    D == 128 ? by_source(std::integral_constant<int, 128>{}) : by_source(std::integral_constant<int, 64>{});
    return check_launch();
}

// What both calls check of the rotation.
qw3_status check_rope(int32_t src_type, int64_t T, int64_t heads, int64_t D, int64_t R, int64_t A, int32_t style) {
    if (src_type != QW3_SRC_BF16 && src_type != QW3_SRC_F32) return QW3_ERR_SHAPE;
    if (style != QW3_ROPE_HALVES && style != QW3_ROPE_PAIRS) return QW3_ERR_SHAPE;
    if (D != 64 && D != 128) return QW3_ERR_SHAPE;
    if (R < 16 || R > D || R % 16 != 0 || A < 1 || A > QW3_MAX_AXES) return QW3_ERR_SHAPE;
    if (heads < 1 || heads > QW3_MAX_HEADS || T < 0 || T >= kMaxGroups) return QW3_ERR_SHAPE;
    return QW3_OK;
}

constexpr int64_t kWidest = int64_t(1) << 32;  // token strides: a row's address stays in 64 bits

}  // namespace

extern "C" {

qw3_status qrope(const void *x, int32_t src_type, const int32_t *positions, const double *rates, const int32_t *axis,
                 int32_t style, uint16_t *out, int64_t T, int64_t H, int64_t D, int64_t R, int64_t A, int64_t x_ts,
                 int64_t x_hs, void *hip_stream) {
    const qw3_status st = check_rope(src_type, T, H, D, R, A, style);
    if (st != QW3_OK) return st;
    if (!strides_ok(x_ts, x_hs, kWidest)) return QW3_ERR_SHAPE;
    if (T == 0) return QW3_OK;
    if (!x || !positions || !rates || !out) return QW3_ERR_NULL;
    const int per = src_type == QW3_SRC_F32 ? 4 : 8;  // elements of 16 bytes
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(positions, 4) || !aligned(rates, 8) || !aligned(axis, 4) ||
        x_ts % per || x_hs % per)
        return QW3_ERR_ALIGN;
    RopeArgs a{};
    a.q = x, a.q_out = out, a.q_ts = x_ts, a.q_hs = x_hs;
    a.positions = positions, a.rates = rates, a.axis = axis;
    a.T = (int)T, a.Hq = (int)H, a.half = (int)(R / 2), a.A = (int)A;
    return launch_rope<false>(a, src_type, QW3_CODES_INT8, D, style, (hipStream_t)hip_stream);
}

qw3_status qrope_write(const void *q, const void *k, const void *v, int32_t src_type, const int32_t *positions,
                       const double *rates, const int32_t *axis, int32_t style, const int64_t *slots, uint16_t *q_out,
                       uint16_t *k_out, uint16_t *v_out, void *codes, float *scales, int32_t code_type, int64_t T,
                       int64_t Hq, int64_t H, int64_t D, int64_t R, int64_t A, int64_t pages, int64_t page_size,
                       int64_t q_ts, int64_t q_hs, int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs,
                       void *hip_stream) {
    int shift = 0;
    qw3_status st = check_cache(code_type, H, D, pages, page_size, &shift);
    if (st != QW3_OK) return st;
    st = check_rope(src_type, T, Hq, D, R, A, style);
    if (st != QW3_OK) return st;
    if (Hq % H != 0 || !strides_ok(q_ts, q_hs, kWidest) || !strides_ok(k_ts, k_hs, kWidest) ||
        !strides_ok(v_ts, v_hs, kWidest))
        return QW3_ERR_SHAPE;
    if (T == 0) return QW3_OK;
    if (!q || !k || !v || !positions || !rates || !slots || !q_out || (pages > 0 && (!codes || !scales)))
        return QW3_ERR_NULL;
    const int per = src_type == QW3_SRC_F32 ? 4 : 8;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) ||
        !aligned(v_out, 16) || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(slots, 8) ||
        !aligned(positions, 4) || !aligned(rates, 8) || !aligned(axis, 4) || q_ts % per || q_hs % per || k_ts % per ||
        k_hs % per || v_ts % per || v_hs % per)
        return QW3_ERR_ALIGN;
    RopeArgs a{};
    a.q = q, a.k = k, a.v = v, a.positions = positions, a.rates = rates, a.axis = axis, a.slots = slots;
    a.q_out = q_out, a.k_out = k_out, a.v_out = v_out, a.codes = static_cast<uint8_t *>(codes), a.scales = scales;
    a.T = (int)T, a.Hq = (int)Hq, a.H = (int)H, a.half = (int)(R / 2), a.A = (int)A, a.page_shift = shift;
    a.n_slots = pages * page_size;
    a.q_ts = q_ts, a.q_hs = q_hs, a.k_ts = k_ts, a.k_hs = k_hs, a.v_ts = v_ts, a.v_hs = v_hs;
    return launch_rope<true>(a, src_type, code_type, D, style, (hipStream_t)hip_stream);
}

}  // extern "C"
