#pragma once
// Device code that the attention kernels share (qw3_attn.hip, qw3_blocks.hip):
// matrix operand types, exchanges between lanes, partial results that pass between
// workgroups, and the cache's codes as bf16.
#include "qw3_quant.h"
#include "qw3_units.h"

using namespace qw3_units;

namespace {

typedef float f16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));
typedef short s4_t __attribute__((ext_vector_type(4)));
typedef short s8_t __attribute__((ext_vector_type(8)));
typedef int i2_t __attribute__((ext_vector_type(2)));
typedef int i4_t __attribute__((ext_vector_type(4)));
#define LDS_AS __attribute__((address_space(3)))

constexpr float kNegInf = -__builtin_huge_valf();
// m may stay this far (in log2) below the true maximum before the sums are
// rescaled: p then reaches at most 2^8, harmless in fp32 and bf16.
constexpr float kSlack = 8.0f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)x);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(x >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ void wait_vm0() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory"); }
// Over the lanes l and l ^ 32 (halves), or l, l ^ 16, l ^ 32, l ^ 48 (quarters).
__device__ __forceinline__ float max_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_quarters(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return max_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float sum_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float sum_quarters(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return sum_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

__device__ __forceinline__ float wave_max_f(float x) {  // over all 64 lanes, in every lane
    for (int d = 8; d >= 1; d /= 2) x = fmaxf(x, __shfl_xor(x, d, 64));
    return max_quarters(x);
}

__device__ __forceinline__ void store_agent(float *p, float x, float y) {
    const uint64_t v = (uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x);
    __hip_atomic_store(reinterpret_cast<uint64_t *>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 load_agent(const float *p) {
    const uint64_t v =
        __hip_atomic_load(reinterpret_cast<const uint64_t *>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}

// By one workgroup of a call that counts: the next call's counters (qw3_units.h).
template <int kThreads>
__device__ __forceinline__ void clear_next(int *counts) {
#pragma unroll
    for (int i = 0; i < kCounts / 2; i += kThreads)
        store_agent(reinterpret_cast<float *>(counts) + 2 * (i + threadIdx.x), 0.0f, 0.0f);
}

__device__ __forceinline__ int wave_sum(int x) {  // over all 64 lanes, in every lane
    x += (int)dpp_u32<0xB1>((uint32_t)x);   // quad_perm [1, 0, 3, 2]
    x += (int)dpp_u32<0x4E>((uint32_t)x);   // quad_perm [2, 3, 0, 1]
    x += (int)dpp_u32<0x141>((uint32_t)x);  // row_half_mirror
    x += (int)dpp_u32<0x140>((uint32_t)x);  // row_mirror
    auto r = __builtin_amdgcn_permlane16_swap((uint32_t)x, (uint32_t)x, false, false);
    x = (int)(r[0] + r[1]);
    r = __builtin_amdgcn_permlane32_swap((uint32_t)x, (uint32_t)x, false, false);
    return (int)(r[0] + r[1]);
}

__device__ __forceinline__ int wave_max(int x) {  // over all 64 lanes, in every lane
    x = max(x, (int)dpp_u32<0xB1>((uint32_t)x));   // as in wave_sum
    x = max(x, (int)dpp_u32<0x4E>((uint32_t)x));
    x = max(x, (int)dpp_u32<0x141>((uint32_t)x));
    x = max(x, (int)dpp_u32<0x140>((uint32_t)x));
    auto r = __builtin_amdgcn_permlane16_swap((uint32_t)x, (uint32_t)x, false, false);
    x = max((int)r[0], (int)r[1]);
    r = __builtin_amdgcn_permlane32_swap((uint32_t)x, (uint32_t)x, false, false);
    return max((int)r[0], (int)r[1]);
}

// Byte J of w, signed, as float.
template <int J>
__device__ __forceinline__ float byte_f32(uint32_t w) {
    float f;
    if (J == 0) asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0" : "=v"(f) : "v"(w));
    if (J == 1) asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1" : "=v"(f) : "v"(w));
    if (J == 2) asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2" : "=v"(f) : "v"(w));
    if (J == 3) asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3" : "=v"(f) : "v"(w));
    return f;
}

// Four codes to four bf16 (two words), exact in both types.
template <bool E4M3>
__device__ __forceinline__ uint2 decode4(uint32_t w) {
    if (E4M3)
        return make_uint2(
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)));
    return make_uint2(pack_bf16(byte_f32<0>(w), byte_f32<1>(w)), pack_bf16(byte_f32<2>(w), byte_f32<3>(w)));
}
template <bool E4M3>
__device__ __forceinline__ bf8_t decode8(uint32_t lo, uint32_t hi) {
    const uint2 a = decode4<E4M3>(lo), b = decode4<E4M3>(hi);
    return __builtin_bit_cast(bf8_t, i4_t{(int)a.x, (int)a.y, (int)b.x, (int)b.y});
}

// Reads of partial results that a wave has under way at once: more of them make
// the code longer, and a call on a short cache waits for its instructions
// (measured with 16 rows: one token over 1000 keys 8.4 us at 16, 9.0 at 32, 10.8
// at 64; with 32 rows trees of 13 want 32: 17.8 us, 18.4 at 16).
template <int R>
constexpr int kFlight = R;

// An item's `rows` rows from the partial results of workgroups first..last in
// that order, by the 4 waves of a workgroup: wave w takes rows w, w + 4, ...
// together, so that their reads, each of which goes to memory, are under way at
// once.  slot_of(g): where workgroup g left its part, R maxima and sums as pairs
// (m, l) and R x D weighted sums.  row_out(r): where row r goes.
template <int R, int D, int kRowsOfWave, class Slot, class RowOut>
__device__ __forceinline__ void join_rows(Slot slot_of, int first, int last, int rows, RowOut row_out) {
    const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
    constexpr int kBatch = kFlight<R> / kRowsOfWave;
    float m[kRowsOfWave], l[kRowsOfWave], f[kRowsOfWave];
    float2 acc[kRowsOfWave];
#pragma unroll
    for (int k = 0; k < kRowsOfWave; ++k) m[k] = kNegInf, l[k] = 0.0f, acc[k] = make_float2(0.0f, 0.0f);
    for (int g0 = first; g0 <= last; g0 += 64) {
        const int n = min(64, last + 1 - g0);
        auto slot = [&](int i) { return slot_of(g0 + i); };
        const float *mine = slot(min(lane, n - 1));
        float2 ml[kRowsOfWave];
#pragma unroll
        for (int k = 0; k < kRowsOfWave; ++k) ml[k] = load_agent(mine + 2 * min(wave + 4 * k, rows - 1));
        float2 part[kBatch][kRowsOfWave];
        auto read = [&](int i0) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const float *p = slot(min(i0 + i, n - 1)) + 2 * R;
#pragma unroll
                for (int k = 0; k < kRowsOfWave; ++k) {
                    const int at = min(wave + 4 * k, rows - 1) * D;
                    if (D == 128)
                        part[i][k] = load_agent(p + at + 2 * lane);
                    else
                        part[i][k].x = __hip_atomic_load(p + at + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                }
            }
        };
        read(0);  // beside the maxima and sums
#pragma unroll
        for (int k = 0; k < kRowsOfWave; ++k) {
            float m1 = lane < n ? ml[k].x : kNegInf;
            for (int x = 32; x >= 1; x /= 2) m1 = fmaxf(m1, __shfl_xor(m1, x, 64));
            m1 = fmaxf(m[k], m1);
            const float old = m[k] == kNegInf ? 0.0f : exp2_fast(m[k] - m1);
            f[k] = lane >= n || ml[k].x == kNegInf ? 0.0f : exp2_fast(ml[k].x - m1);
            float ls = f[k] == 0.0f ? 0.0f : f[k] * ml[k].y;
            for (int x = 32; x >= 1; x /= 2) ls += __shfl_xor(ls, x, 64);
            m[k] = m1;
            l[k] = l[k] * old + ls;
            acc[k].x *= old, acc[k].y *= old;
        }
        for (int i0 = 0; i0 < n; i0 += kBatch) {
            if (i0 > 0) read(i0);
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
#pragma unroll
                for (int k = 0; k < kRowsOfWave; ++k) {
                    const float fi = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f[k]), min(i0 + i, n - 1)));
                    if (i0 + i < n) {
                        acc[k].x += fi * part[i][k].x;
                        if (D == 128) acc[k].y += fi * part[i][k].y;
                    }
                }
        }
    }
#pragma unroll
    for (int k = 0; k < kRowsOfWave; ++k) {
        if (wave + 4 * k >= rows) continue;
        const float inv = l[k] == 0.0f ? 0.0f : 1.0f / l[k];
        uint16_t *out = row_out(wave + 4 * k);
        if (D == 128)
            *reinterpret_cast<uint32_t *>(out + 2 * lane) = pack_bf16(acc[k].x * inv, acc[k].y * inv);
        else
            out[lane] = (uint16_t)(pack_bf16(acc[k].x * inv, 0.0f) & 0xffffu);
    }
}

}  // namespace
