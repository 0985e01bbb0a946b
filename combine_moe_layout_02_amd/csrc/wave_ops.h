// Reductions over the 64 lanes of a wave whose result every lane has, in a fixed order: four steps inside a row of 16 lanes
// through DPP, two between the rows through the lane swaps, none through LDS (a shuffle is an LDS access, of some 100
// cycles a step).
#pragma once

#include "moe_internal.h"

namespace moe {
namespace wave {

template <int CTRL>
__device__ inline uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

constexpr int kQuadSwap1 = 0xB1, kQuadSwap2 = 0x4E;       // quad_perm 1,0,3,2 and 2,3,0,1
constexpr int kRowHalfMirror = 0x141, kRowMirror = 0x140;  // lane i of 8, of 16, from 7 - i, 15 - i

// The value of the lane across (kind) as the same type: after the steps before, a lane and its mirror's neighbours
// hold the same, so that mirrors do as well as exchanges.
template <int CTRL>
__device__ inline float across(float v) { return __uint_as_float(dpp<CTRL>(__float_as_uint(v))); }
template <int CTRL>
__device__ inline int across(int v) { return (int)dpp<CTRL>((uint32_t)v); }
template <int CTRL>
__device__ inline uint32_t across(uint32_t v) { return dpp<CTRL>(v); }
template <int CTRL>
__device__ inline double across(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)b) | (uint64_t)dpp<CTRL>((uint32_t)(b >> 32)) << 32);
}

// Both halves of an exchange between neighbouring rows (ROWS) or between the wave's halves: in every lane the one is the
// own group's value and the other the group's across, in the same order everywhere.
template <bool ROWS>
__device__ inline void swap(uint32_t v, uint32_t &a, uint32_t &b) {
    if constexpr (ROWS) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        a = r[0], b = r[1];
    } else {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        a = r[0], b = r[1];
    }
}

template <bool ROWS, class T, class OP>
__device__ inline T join(T v, OP op) {
    if constexpr (sizeof(T) == 4) {
        uint32_t a, b;
        swap<ROWS>(__builtin_bit_cast(uint32_t, v), a, b);
        return op(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));
    } else {
        const uint64_t bits = __builtin_bit_cast(uint64_t, v);
        uint32_t alo, blo, ahi, bhi;
        swap<ROWS>((uint32_t)bits, alo, blo);
        swap<ROWS>((uint32_t)(bits >> 32), ahi, bhi);
        return op(__builtin_bit_cast(T, (uint64_t)alo | (uint64_t)ahi << 32), __builtin_bit_cast(T, (uint64_t)blo | (uint64_t)bhi << 32));
    }
}

template <class T, class OP>
__device__ inline T reduce(T v, OP op) {
    v = op(v, across<kQuadSwap1>(v));
    v = op(v, across<kQuadSwap2>(v));
    v = op(v, across<kRowHalfMirror>(v));
    v = op(v, across<kRowMirror>(v));
    v = join<true>(v, op);
    return join<false>(v, op);
}

template <class T>
__device__ inline T sum(T v) {
    return reduce(v, [](T a, T b) { return a + b; });
}
__device__ inline uint32_t most(uint32_t v) {
    return reduce(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ inline float most(float v) {
    return reduce(v, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace wave
}  // namespace moe
