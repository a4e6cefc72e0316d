// mx.h -- microscaled 4-bit floating point (MXFP4) in device code: blocks of 32
// consecutive values with one E8M0 byte b, scale 2^(b - 127), and an E2M1 code
// each (0, 0.5, 1, 1.5, 2, 3, 4, 6, sign in bit 3), the even value in a byte's
// low half.
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kMxBlock = 32;

// The E8M0 byte of a block whose largest magnitude has the fp32 bits `amax`: the
// largest magnitude's power of two over 4, the largest code's, and 2^-127 at the
// least; 255 (not a number) for a block with a NaN or an infinity, whose bits are
// the largest as integers.
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax)
{
    const uint32_t e = amax >> 23;
    return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// The instructions' scale operands take an E8M0 byte as a float's exponent, 0
// meaning 2^-127 and 255 not a number.
__device__ __forceinline__ float mx_scale_operand(uint32_t b) { return __uint_as_float(b << 23); }

// Magnitude bits of x.
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Eight E2M1 codes of x / 2^(b - 127), nearest, ties to even, at most 6 in
// magnitude, the first in the lowest four bits; zeros for b = 255.
__device__ __forceinline__ uint32_t mx_pack8(const float (&x)[8], uint32_t b)
{
    const float s = mx_scale_operand(b);
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[0], x[1], s, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[2], x[3], s, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[4], x[5], s, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[6], x[7], s, 3);
    return b == 255u ? 0u : q;
}

// The largest value over the four lanes that a block of 32 is spread over (8
// values each).
__device__ __forceinline__ uint32_t max_of_quad(uint32_t m)
{
    // quad_perm 1 0 3 2, then 2 3 0 1
    m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0xB1, 0xF, 0xF, true)));
    return max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0x4E, 0xF, 0xF, true)));
}

// The bytes of lanes 0, 4, 8 and 12 of each group of 16 as one word, in all of
// them.
__device__ __forceinline__ uint32_t gather_bytes(uint32_t b)
{
    return __shfl(b, 0, 16) | (__shfl(b, 4, 16) << 8) | (__shfl(b, 8, 16) << 16) | (__shfl(b, 12, 16) << 24);
}

}  // namespace moe
