// OCP FP8 E4M3 helpers shared by the quantising kernels (gfx950).
#pragma once

#include "common.h"

namespace moe {

// Exponent e of the scale 2^e of a row or block: the smallest integer with
// amax <= 448 * 2^e (0 for amax == 0).  With amax = m * 2^x, m in [0.5, 1):
// 448 = 0.875 * 2^9, so e = x - 9 when m <= 0.875, else x - 8.
__device__ __forceinline__ int fp8_scale_exp(float amax)
{
    if (!(amax > 0.0f))
        return 0;
    int x;
    const float m = frexpf(amax, &x);
    return m <= 0.875f ? x - 9 : x - 8;
}

// E4M3 codes of 8 values scaled by 2^-e (|f / 2^e| <= 448), little-endian
// bytes in value order.
__device__ __forceinline__ uint2 e4m3_encode8(const float* f, int e)
{
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(f[0], -e), ldexpf(f[1], -e), 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(f[2], -e), ldexpf(f[3], -e), lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(f[4], -e), ldexpf(f[5], -e), 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(f[6], -e), ldexpf(f[7], -e), hi, true);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// Exponent of an E8M0 block scale (the byte e + 127 stands for 2^e): the
// smallest e with amax <= 448 * 2^e that the byte can hold.
__device__ __forceinline__ int fp8_block_scale_exp(float amax)
{
    return min(max(fp8_scale_exp(amax), -127), 127);
}

}  // namespace moe
