// The quantised key/value cache: rows are quantised as they are written
// (qcache_write) and read back dense (qcache_read).  C ABI in include/qw3.h.
//
// One row is what one token stores for one kv head: D channels x_d with one
// fp32 scale s.  a = max |x_d|, s = a / L, c_d = rne(x_d / s), L = 127 for
// int8 codes and 448 for e4m3; the row stands for c_d s.  Both divisions are
// IEEE divisions in fp32, so the codes do not depend on how the work is laid
// out.  Both operations are bound by memory: 8191 tokens of 8 heads of 128
// channels, bf16 to e4m3, are written in 11 us (4.5 TB/s) and read back in 10,
// 60,000 tokens read in 119 us (4.8 TB/s; a large copy reaches 4.9).
#include "qw3_common.h"

using namespace qw3_shared;

namespace {

typedef float f2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bfx2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const f2_t f = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bfx2_t));
}

// ------------------------------------------------------------------ write --
// A row is quantised by D / 16 lanes of one wave, 16 channels each; a workgroup
// has consecutive tokens of one head, keys and values, so its loads and stores
// are whole rows, no lane divides to find its row, and both rows' loads are on
// their way together.  Neighbouring workgroups have the heads of the same tokens:
// what the card reads at one time lies together in memory.
//
// The quotients.  A row's 128 divisions by the same s cost more than all else
// here.  With r the correctly rounded 1 / s, one division for the row, each
// quotient is refined by its exact remainder: q = x r; q += (x - q s) r makes it
// one of the two floats around x / s; q += (x - q s) r the correctly rounded one
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990), where neither r nor a remainder leaves the normal numbers:
// rows with s outside 2^-80..2^100 divide.  So codes are those of the IEEE
// quotient for every input.
template <bool E4M3>
__device__ __forceinline__ uint32_t codes4(const float (&y)[4]) {
    if (E4M3) {
        const int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
    }
    // 1.5 2^23 + y is rounded to a whole number, whose two's complement is its low byte
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(y[i] + 12582912.0f);
    const uint32_t lo = __builtin_amdgcn_perm(w[1], w[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(w[3], w[2], 0x04000c0cu);
    return lo | hi;
}

template <bool F32>
struct Source {
    uint4 w[F32 ? 4 : 2];
    __device__ __forceinline__ void load(const void *p, int64_t at, int c) {
        const uint4 *src = F32 ? reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + at)
                               : reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at);
#pragma unroll
        for (int i = 0; i < (F32 ? 4 : 2); ++i) w[i] = src[(F32 ? 4 : 2) * c + i];
    }
    __device__ __forceinline__ void values(float (&x)[16]) const {
#pragma unroll
        for (int i = 0; i < (F32 ? 4 : 2); ++i) {
            const uint32_t d[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (F32) {
                    x[4 * i + e] = __uint_as_float(d[e]);
                } else {
                    x[8 * i + 2 * e] = __uint_as_float(d[e] << 16);
                    x[8 * i + 2 * e + 1] = __uint_as_float(d[e] & 0xffff0000u);
                }
            }
        }
    }
};

template <int D, bool F32, bool E4M3>
__device__ __forceinline__ float quantise(const Source<F32> &src, uint32_t (&out)[4]) {
    constexpr int kLanes = D / 16;
    constexpr float kLimit = E4M3 ? 448.0f : 127.0f;
    float x[16];
    src.values(x);
    // |x| as bits orders like the value, with infinities and NaN on top
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
    for (int m = kLanes / 2; m >= 1; m /= 2) top = max(top, (uint32_t)__shfl_xor((int)top, m, 64));
    const bool finite = top < 0x7f800000u;
    const float s = finite ? __uint_as_float(top) / kLimit : __uint_as_float(0x7fc00000u);
    if (s > 0x1p-80f && s < 0x1p100f) {
        const float r = 1.0f / s;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float v = x[4 * i + e];
                float q = v * r;
                q = fmaf(fmaf(-q, s, v), r, q);
                y[e] = fmaf(fmaf(-q, s, v), r, q);
            }
            out[i] = codes4<E4M3>(y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y[4];
            // past L only where s is a denormal and a / L was rounded down; no s, no codes
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = s > 0.0f ? fminf(fmaxf(x[4 * i + e] / s, -kLimit), kLimit) : 0.0f;
            out[i] = codes4<E4M3>(y);
        }
    }
    return s;
}

template <int D, bool F32, bool E4M3>
__global__ __launch_bounds__(256) void cache_write_kernel(const void *__restrict__ k, const void *__restrict__ v,
                                                          const int64_t *__restrict__ slots,
                                                          uint8_t *__restrict__ codes, float *__restrict__ scales,
                                                          int T, int H, int page_shift, int64_t n_slots, int64_t k_ts,
                                                          int64_t k_hs, int64_t v_ts, int64_t v_hs) {
    constexpr int kLanes = D / 16;
    const int group = (int)(blockIdx.x / (uint32_t)H), h = (int)blockIdx.x - group * H;
    const int t = group * (256 / kLanes) + threadIdx.x / kLanes, c = threadIdx.x % kLanes;
    // every lane of a row takes the same branch, so the row's exchanges stay whole
    if (t >= T) return;
    const int64_t slot = slots[t];
    Source<F32> kx, vx;
    kx.load(k, t * k_ts + h * k_hs, c);
    vx.load(v, t * v_ts + h * v_hs, c);
    if (slot < 0 || slot >= n_slots) return;
    const int64_t page = slot >> page_shift;
    const int64_t at = ((page * 2 * H + h) << page_shift) + (slot - (page << page_shift));
    const int64_t to_v = (int64_t)H << page_shift;
    uint32_t out[4];
    const float ks = quantise<D, F32, E4M3>(kx, out);
    reinterpret_cast<uint4 *>(codes + at * D)[c] = make_uint4(out[0], out[1], out[2], out[3]);
    if (c == 0) scales[at] = ks;
    const float vs = quantise<D, F32, E4M3>(vx, out);
    reinterpret_cast<uint4 *>(codes + (at + to_v) * D)[c] = make_uint4(out[0], out[1], out[2], out[3]);
    if (c == 0) scales[at + to_v] = vs;
}

// ------------------------------------------------------------------- read --
// A workgroup reads 16 consecutive rows of the packed output for every head,
// of the keys or of the values; lanes run over a row's 16-byte pieces, then
// over the tokens, so loads follow a page's tokens.  kAtOnce heads' rows are on
// their way together: 4 for many rows (60,000 tokens of 8 heads 119 us, 128 with
// 1), 1 where a CU has only a few workgroups (8191 tokens 10 us, 11 with 4).
template <int D, bool E4M3, int kAtOnce>
__global__ __launch_bounds__(256) void cache_read_kernel(const uint8_t *__restrict__ codes,
                                                         const float *__restrict__ scales,
                                                         const int32_t *__restrict__ table,
                                                         const int32_t *__restrict__ cu, uint16_t *__restrict__ k_out,
                                                         uint16_t *__restrict__ v_out, int B, int64_t max_pages,
                                                         int64_t pages, int64_t total, int H, int page_shift) {
    constexpr int kPieces = D / 16;
    const int lane = threadIdx.x & 63, which = blockIdx.y;
    const int64_t t0 = (int64_t)blockIdx.x * 16;
    // b: the first sequence that ends past t; start: the largest start up to its own
    int b = 0, start = cu[0];
    for (int base = 0; base < B; base += 64) {
        const int end = base + lane < B ? cu[base + lane + 1] : 0x7fffffff;
        const unsigned long long past = __ballot(end > t0);
        const int n = past ? __builtin_ctzll(past) : 64;
        int top = n > 0 ? __builtin_amdgcn_readlane(end, n - 1) : start;
        if (__any(lane < n && end > top)) {  // starts that fall
            top = lane < n ? end : start;
            for (int m = 32; m >= 1; m /= 2) top = max(top, __shfl_xor(top, m, 64));
        }
        start = max(start, top);
        b += n;
        if (past) break;
    }
    const int tok = (threadIdx.x / kPieces) & 15, piece = threadIdx.x % kPieces;
    const int64_t t = t0 + tok;
    for (; b < B; ++b) {
        const int end = cu[b + 1];
        if (end > t) break;
        start = max(start, end);
    }
    if (b >= B || t >= total) return;
    const int64_t pos = t - start, idx = pos >> page_shift;
    if (pos < 0) return;
    int64_t page = idx < max_pages ? table[b * max_pages + idx] : -1;
    const bool there = page >= 0 && page < pages;
    if (!there) page = 0;
    const int64_t row0 = ((page * 2 + which) * H << page_shift) + (pos & ((int64_t(1) << page_shift) - 1));
    uint16_t *out = (which ? v_out : k_out) + t * H * D + piece * 16;
    constexpr int kStep = 256 / (16 * kPieces);
    for (int h0 = threadIdx.x / (16 * kPieces); h0 < H; h0 += kStep * kAtOnce) {
        uint4 c[kAtOnce];
        float s[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int64_t row = row0 + ((int64_t)(h0 + kStep * i) << page_shift);
            c[i] = make_uint4(0, 0, 0, 0), s[i] = 0.0f;
            if (there && h0 + kStep * i < H) {
                c[i] = *reinterpret_cast<const uint4 *>(codes + row * D + piece * 16);
                s[i] = scales[row];
            }
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float f[4];
                if (E4M3) {
                    f[0] = __builtin_amdgcn_cvt_f32_fp8(w[j], 0), f[1] = __builtin_amdgcn_cvt_f32_fp8(w[j], 1);
                    f[2] = __builtin_amdgcn_cvt_f32_fp8(w[j], 2), f[3] = __builtin_amdgcn_cvt_f32_fp8(w[j], 3);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] = (float)(int8_t)(w[j] >> (8 * e));
                }
                o[2 * j] = pack_bf16(f[0] * s[i], f[1] * s[i]);
                o[2 * j + 1] = pack_bf16(f[2] * s[i], f[3] * s[i]);
            }
            if (h0 + kStep * i < H) {
                uint4 *dst = reinterpret_cast<uint4 *>(out + (int64_t)(h0 + kStep * i) * D);
                dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
                dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
            }
        }
    }
}

}  // namespace

extern "C" {

qw3_status qcache_write(const void *k, const void *v, int32_t src_type, const int64_t *slots, void *codes,
                        float *scales, int32_t code_type, int64_t T, int64_t H, int64_t D, int64_t pages,
                        int64_t page_size, int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs, void *hip_stream) {
    int shift = 0;
    const qw3_status st = check_cache(code_type, H, D, pages, page_size, &shift);
    if (st != QW3_OK) return st;
    if (src_type != QW3_SRC_BF16 && src_type != QW3_SRC_F32) return QW3_ERR_SHAPE;
    if (T < 0 || T > QW3_MAX_TOKENS) return QW3_ERR_SHAPE;
    const int64_t groups = ceil_div(T, 256 / (D / 16)) * H;
    if (groups >= kMaxGroups) return QW3_ERR_SHAPE;
    const int64_t widest = int64_t(1) << 32;  // a row's address stays in 64 bits
    if (!strides_ok(k_ts, k_hs, widest) || !strides_ok(v_ts, v_hs, widest)) return QW3_ERR_SHAPE;
    if (T == 0 || pages == 0) return QW3_OK;
    if (!k || !v || !slots || !codes || !scales) return QW3_ERR_NULL;
    const int per = src_type == QW3_SRC_F32 ? 4 : 8;  // elements of 16 bytes
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(slots, 8) ||
        k_ts % per || k_hs % per || v_ts % per || v_hs % per)
        return QW3_ERR_ALIGN;
    const dim3 grid((unsigned)groups);
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, (hipStream_t)hip_stream, k, v, slots, (uint8_t *)codes, scales,
                           (int)T, (int)H, shift, pages * page_size, k_ts, k_hs, v_ts, v_hs);
    };
    auto by_type = [&](auto d) {
        constexpr int kD = decltype(d)::value;
        if (src_type == QW3_SRC_F32)
            code_type == QW3_CODES_E4M3 ? run(cache_write_kernel<kD, true, true>)
                                        : run(cache_write_kernel<kD, true, false>);
        else
            code_type == QW3_CODES_E4M3 ? run(cache_write_kernel<kD, false, true>)
                                        : run(cache_write_kernel<kD, false, false>);
    };
    D == 128 ? by_type(std::integral_constant<int, 128>{}) : by_type(std::integral_constant<int, 64>{});
    return check_launch();
}

qw3_status qcache_read(const void *codes, const float *scales, int32_t code_type, const int32_t *block_table,
                       const int32_t *cu, uint16_t *k_out, uint16_t *v_out, int64_t B, int64_t max_pages,
                       int64_t total, int64_t H, int64_t D, int64_t pages, int64_t page_size, void *hip_stream) {
    int shift = 0;
    const qw3_status st = check_cache(code_type, H, D, pages, page_size, &shift);
    if (st != QW3_OK) return st;
    if (B < 0 || B > QW3_MAX_SEQS || max_pages < 0 || total < 0 || total > QW3_MAX_TOKENS)
        return QW3_ERR_SHAPE;
    if (B == 0 || total == 0) return QW3_OK;
    if (!cu || !k_out || !v_out || (max_pages > 0 && !block_table) || (pages > 0 && (!codes || !scales)))
        return QW3_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(block_table, 4) || !aligned(cu, 4) ||
        !aligned(k_out, 16) || !aligned(v_out, 16))
        return QW3_ERR_ALIGN;
    const dim3 grid((unsigned)ceil_div(total, 16), 2);
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, (hipStream_t)hip_stream, (const uint8_t *)codes, scales,
                           block_table, cu, k_out, v_out, (int)B, max_pages, pages, total, (int)H, shift);
    };
    auto by_size = [&](auto d, auto type) {
        constexpr int kD = decltype(d)::value;
        constexpr bool kType = decltype(type)::value;
        total >= 16384 ? run(cache_read_kernel<kD, kType, 4>) : run(cache_read_kernel<kD, kType, 1>);
    };
    auto by_type = [&](auto d) {
        code_type == QW3_CODES_E4M3 ? by_size(d, std::true_type{}) : by_size(d, std::false_type{});
    };
    D == 128 ? by_type(std::integral_constant<int, 128>{}) : by_type(std::integral_constant<int, 64>{});
    return check_launch();
}

}  // extern "C"
