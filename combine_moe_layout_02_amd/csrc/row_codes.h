// Eight fp32 values to 8-bit codes with their row's scale: the codes of the correctly rounded quotients value / scale, as
// pack_rows.h has them for the dispatch, with less around the quotients. No value is larger than top * scale but for the
// scale's rounding, so a quotient is at most top + ulp and its code needs no clamp; adding 1.5 * 2^23 rounds an INT8 quotient to
// a whole number, to even, in the low byte; and its zeros need no sign.
#pragma once

#include "mx_blocks.h"
#include "pack_rows.h"

namespace moe {
namespace rows {

// Codes by the IEEE division, for scales that the corrections do not reach.
template <int QUANT>
__device__ inline mx::u32x2 divided8(const float (&v)[8], float scale) {
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = v[e] / scale;
    if constexpr (QUANT == MOE_QUANT_FP8_E4M3_DYN)
        return mx::u32x2{e4m3fn_pack4(q[0], q[1], q[2], q[3]), e4m3fn_pack4(q[4], q[5], q[6], q[7])};
    mx::u32x2 c;
#pragma unroll
    for (int w = 0; w < 2; ++w)
        c[w] = int8_code(q[4 * w]) | (int8_code(q[4 * w + 1]) << 8) | (int8_code(q[4 * w + 2]) << 16) | (int8_code(q[4 * w + 3]) << 24);
    return c;
}

// Codes by div_by_scale's corrections, inv = RN(1 / scale).
template <int QUANT>
__device__ inline mx::u32x2 codes8(const float (&v)[8], float scale, float inv) {
    mx::u32x2 c;
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q0 = v[e] * inv, q1 = __builtin_fmaf(__builtin_fmaf(-q0, scale, v[e]), inv, q0);
        q[e] = __builtin_fmaf(__builtin_fmaf(-q1, scale, v[e]), inv, q1);
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        if constexpr (QUANT == MOE_QUANT_INT8_DYN) {
            constexpr float kWhole = 12582912.0f;
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] = __float_as_uint(q[4 * w + e] + kWhole);
            const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400), hi = __builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400);
            c[w] = __builtin_amdgcn_perm(hi, lo, 0x05040100);
        } else {
#pragma unroll
            for (int e = 4 * w; e < 4 * w + 4; ++e) q[e] = __builtin_copysignf(q[e], v[e]);
            int p = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * w], q[4 * w + 1], 0, false);
            p = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * w + 2], q[4 * w + 3], p, true);
            c[w] = (uint32_t)p;
        }
    }
    return c;
}

// RN(1 / scale) and the corrections give the correctly rounded quotient unless all bits of the scale's mantissa are set; below
// kFastDivMinScale a remainder may leave the normal range.
__device__ inline bool corrected(float scale) {
    return scale >= kFastDivMinScale && scale <= 0x1.fffffep127f && (__float_as_uint(scale) & 0x7FFFFFu) != 0x7FFFFFu;
}

}  // namespace rows
}  // namespace moe
