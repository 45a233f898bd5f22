// MXFP4 helpers (gfx950): E2M1 codes (sign, 2 exponent bits, 1 mantissa bit:
// 0, 0.5, 1, 1.5, 2, 3, 4, 6) with an E8M0 scale for each block of 32 values.
#pragma once

#include "common.h"

namespace moe {

constexpr int kMxBlk = 32;        // values that share a scale
constexpr uint32_t kMxNan = 255;  // the scale byte of a block that holds a NaN or an infinity

// |f| as an integer that orders finite values, infinity and NaNs, in this order.
__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7fffffffu; }

// Scale byte e + 127 of a block whose largest |value| has these bits: the
// smallest e >= -127 with amax <= 6 * 2^e (0 for an all-zero block).  With amax =
// m * 2^x, m in [0.5, 1): 6 = 0.75 * 2^3, so e = x - 3 when m <= 0.75, else x - 2.
// E2M1 has no NaN: a block with a NaN or an infinity becomes NaN as a whole.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax)
{
    if (amax >= 0x7f800000u)
        return kMxNan;
    if (amax == 0)
        return 127;
    int x;
    const float m = frexpf(__uint_as_float(amax), &x);
    return (uint32_t)(max(m <= 0.75f ? x - 3 : x - 2, -127) + 127);
}

// E2M1 codes of 8 values of a block with scale byte s, nearest to v / 2^(s - 127),
// ties to the even code; the first value in the lowest four bits.  v / 2^e is
// exact, so every code is decided exactly.  A NaN block gets codes of 6.
__device__ __forceinline__ uint32_t e2m1_encode8(const float* f, uint32_t s)
{
    if (s == kMxNan)
        return 0x77777777u;
    const int e = (int)s - 127;
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, ldexpf(f[0], -e), ldexpf(f[1], -e), 1.0f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, ldexpf(f[2], -e), ldexpf(f[3], -e), 1.0f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, ldexpf(f[4], -e), ldexpf(f[5], -e), 1.0f, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, ldexpf(f[6], -e), ldexpf(f[7], -e), 1.0f, 3);
}

// The 8 values that codes c stand for in a block with scale byte s.
__device__ __forceinline__ void e2m1_decode8(uint32_t c, uint32_t s, float* f)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
    const f32x2 g = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y, f[4] = d.x, f[5] = d.y, f[6] = g.x, f[7] = g.y;
    const int e = (int)s - 127;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = s == kMxNan ? __builtin_nanf("") : ldexpf(f[i], e);
}

}  // namespace moe
