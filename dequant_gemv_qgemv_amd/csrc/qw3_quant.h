#pragma once
// Quantising a row of the key/value cache: shared by the kernels that write it.
// One row is what one token stores for one kv head: D channels x_d with one fp32
// scale s.  a = max |x_d|, s = a / L, c_d = rne(x_d / s), L = 127 for int8 codes
// and 448 for e4m3.
#include "qw3_common.h"

namespace {

typedef float f2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const f2_t f = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf2_t));
}

// The quotients.  A row's 128 divisions by the same s cost more than all else of
// a kernel that writes it.  With r the correctly rounded 1 / s, one division for
// the row, each quotient is refined by its exact remainder: q = x r; q += (x - q s) r makes it
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

// Of a row's D channels the lane's 16, whatever they are: their codes, four in a
// word, and the row's scale.  Its D / 16 lanes are neighbours.
template <int D, bool E4M3>
__device__ __forceinline__ float quantise(const float (&x)[16], uint32_t (&out)[4]) {
    constexpr int kLanes = D / 16;
    constexpr float kLimit = E4M3 ? 448.0f : 127.0f;
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

}  // namespace
