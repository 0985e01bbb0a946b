// Device helpers for MX blocks (OCP Microscaling specification, version 1.0): the scale byte of 32 bf16
// values, and codes and values of eight of them at a time, the share of one lane.
//
// A block's byte comes from its largest magnitude as bf16 bits, amax = 1.M * 2^(E - 127) (0.M * 2^-126 for
// E = 0):
//   E2M1: floor(log2(amax)) - 2, so byte = max(E - 2, 0);
//   E4M3: the smallest e with amax <= 448 * 2^e = 1.75 * 2^(e + 8): E - 127 - 8, or one more where 1.M > 1.75
//         (M > 96), so byte = max(E - 8 + (M > 96), 0).
// Both hold for E = 0 and a zero block, where the byte is 0. x * 2^(127 - byte) is exact in fp32 unless it
// falls below fp32's normal range, which rounds to a zero code either way; the one rounding is the
// hardware's conversion to the code (to nearest even; E2M1 saturates at 6, E4M3 never exceeds 448 here).
#pragma once

#include "moe_internal.h"

namespace moe {
namespace mx {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kNanByte = 255;

__device__ inline float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ inline float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two fp32 values to bf16, to nearest even, in one word.
__device__ inline uint32_t bf16_pair(float lo, float hi) {
    const bf16x2 p = __builtin_convertvector((f32x2{lo, hi}), bf16x2);
    return __builtin_bit_cast(uint32_t, p);
}

// Largest magnitude of eight bf16 values, as bf16 bits.
__device__ inline uint32_t amax_bits(const u32x4 &v) {
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        m = max(m, v[w] & 0x7FFFu);
        m = max(m, (v[w] >> 16) & 0x7FFFu);
    }
    return m;
}

// The largest over each four neighbouring lanes (one block of 32 values), in all four.
__device__ inline uint32_t max_of_four_lanes(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));  // quad_perm 1,0,3,2
    return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));  // 2,3,0,1
}

// The scale byte for a block's largest magnitude; 255 where it is an infinity or a NaN.
template <int FORMAT>
__device__ inline uint32_t scale_byte(uint32_t amax) {
    const int e = (int)(amax >> 7);
    if (e == 255) return kNanByte;
    if constexpr (FORMAT == MOE_MX_E2M1) return (uint32_t)max(e - 2, 0);
    else return (uint32_t)max(e - 8 + ((amax & 0x7Fu) > 96u ? 1 : 0), 0);
}

// What a scale byte is worth (2^-127 is an fp32 subnormal, 255 a NaN).
__device__ inline float scale_value(uint32_t byte) {
    const uint32_t bits = byte == 0 ? 0x00400000u : byte == kNanByte ? 0x7FC00000u : byte << 23;
    return __uint_as_float(bits);
}

// 2^(127 - byte), what a block's values are multiplied by (byte <= 252 for any finite block).
__device__ inline float inverse_scale(uint32_t byte) {
    return __uint_as_float((254u - byte) << 23);
}

// Codes of eight bf16 values: one word (E2M1) or two (E4M3), in element order; zero for byte 255.
template <int FORMAT>
__device__ inline u32x2 encode(const u32x4 &v, uint32_t byte) {
    if (byte == kNanByte) return u32x2{0u, 0u};
    const float inv = inverse_scale(byte);
    if constexpr (FORMAT == MOE_MX_E2M1) {
        uint32_t r = 0;
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, bf16_lo(v[0]) * inv, bf16_hi(v[0]) * inv, 1.0f, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, bf16_lo(v[1]) * inv, bf16_hi(v[1]) * inv, 1.0f, 1);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, bf16_lo(v[2]) * inv, bf16_hi(v[2]) * inv, 1.0f, 2);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, bf16_lo(v[3]) * inv, bf16_hi(v[3]) * inv, 1.0f, 3);
        return u32x2{r, 0u};
    } else {
        u32x2 r;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            int p = __builtin_amdgcn_cvt_pk_fp8_f32(bf16_lo(v[2 * w]) * inv, bf16_hi(v[2 * w]) * inv, 0, false);
            p = __builtin_amdgcn_cvt_pk_fp8_f32(bf16_lo(v[2 * w + 1]) * inv, bf16_hi(v[2 * w + 1]) * inv, p, true);
            r[w] = (uint32_t)p;
        }
        return r;
    }
}

// The values of eight E4M3 codes times the scale: a product with a power of two, exact but for results
// below fp32's normal range.
__device__ inline void decode_e4m3(u32x2 codes, float scale, float (&v)[8]) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[w], false);
        const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[w], true);
        v[4 * w] = a.x * scale;
        v[4 * w + 1] = a.y * scale;
        v[4 * w + 2] = b.x * scale;
        v[4 * w + 3] = b.y * scale;
    }
}

// The same for eight E2M1 codes.
__device__ inline void decode_e2m1(uint32_t codes, float scale, float (&v)[8]) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3);
    v[0] = a.x * scale; v[1] = a.y * scale;
    v[2] = b.x * scale; v[3] = b.y * scale;
    v[4] = c.x * scale; v[5] = c.y * scale;
    v[6] = d.x * scale; v[7] = d.y * scale;
}

}  // namespace mx
}  // namespace moe
