// Device helpers of the microscaled 4-bit format (OCP MXFP4): e2m1 codes, two a
// byte with the even column in the low half, and one E8M0 scale (2^(byte - 127),
// 255 = NaN) for each 32 consecutive values of a row.
#pragma once

#include "common.h"

namespace moe {
namespace {

// Scale byte of a block from the bits of its largest magnitude: that magnitude's
// exponent less 2, the exponent of the largest code (6), at least -127.  Taken as
// integers, so that a NaN counts as the largest; NaN and infinity give 255.
__device__ __forceinline__ uint32_t mxfp4_scale(uint32_t amax_bits)
{
    const uint32_t e = amax_bits >> 23;
    return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// Eight codes of v / 2^(scale - 127), v[0] in the low half-byte: rounded to
// nearest, ties to the even code, saturating at 6 (checked on gfx950 at every
// midpoint and its neighbours, from subnormal scales to the largest).  The
// conversions read the exponent field of their scale operand alone.
__device__ __forceinline__ uint32_t mxfp4_codes(const float (&v)[8], uint32_t scale)
{
    const float s = __uint_as_float(scale << 23);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
    return w;
}

// The eight bf16 values that a word of codes stands for: exact but past bf16's
// range (an infinity); NaN for scale 255.
__device__ __forceinline__ u32x4_t mxfp4_to_bf16x8(uint32_t w, uint32_t scale)
{
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    const float s = __uint_as_float(scale << 23);
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
    const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
    return u32x4_t{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                   __builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, d)};
}

}  // namespace
}  // namespace moe
