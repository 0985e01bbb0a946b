// Device helpers shared by the experts' products (mx_product.hip, int8_product.hip): the groups' rows and tiles, the
// gated activation, loads straight to LDS and the barrier between stages.
#pragma once

#include "mx_blocks.h"

namespace moe {
namespace product {

using namespace mx;

typedef int i32x4 __attribute__((ext_vector_type(4)));

// The rows [lo, hi) of groups g0 .. g0 + 63, one a lane (none past the last group). A base below an earlier one
// counts as that one, so that the groups' rows are disjoint and their tiles as many as the grid's arithmetic assumes,
// whatever the bases are. `reached` is where the groups before g0 end, and then where these do. Every lane of a
// wave calls this; bases that ascend, the same for the whole wave, need no running maximum.
__device__ inline void group_rows(const int32_t *__restrict__ base, int G, int a_rows, int g0, int &reached, int &lo,
                                  int &hi) {
    const int lane = threadIdx.x & 63;
    lo = min(max(base[min(g0 + lane, G)], 0), a_rows);
    hi = min(max(base[min(g0 + lane + 1, G)], 0), a_rows);
    if (__any(hi < lo || lo < reached)) {
        hi = max(hi, lo);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int u = __shfl_up(hi, d, 64);
            if (lane >= d) hi = max(hi, u);
        }
        hi = max(hi, reached);
        const int prev = __shfl_up(hi, 1, 64);
        lo = max(lo, lane > 0 ? prev : reached);
    }
    reached = __shfl(hi, 63, 64);
}

// The rows [first, last) that tile number `tile` covers, TM rows at most, and their group; false when there
// are fewer tiles. Groups' tiles follow one another; every lane of a wave calls this and gets the same.
template <int TM>
__device__ inline bool find_rows(const int32_t *__restrict__ base, int G, int64_t a_rows, int tile,
                                 int &group, int64_t &first, int64_t &last) {
    const int lane = threadIdx.x & 63;
    int before = 0, reached = 0;
    for (int g0 = 0; g0 < G; g0 += 64) {
        int lo, hi;
        group_rows(base, G, (int)a_rows, g0, reached, lo, hi);
        const int tiles = (hi - lo + TM - 1) / TM;
        int incl = tiles;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int u = __shfl_up(incl, d, 64);
            if (lane >= d) incl += u;
        }
        const uint64_t here = __ballot(tile < before + incl);  // the group is the first such lane
        if (here) {
            const int src = __ffsll((unsigned long long)here) - 1;
            const int skipped = before + __shfl(incl - tiles, src, 64);
            const int64_t glo = __shfl(lo, src, 64), ghi = __shfl(hi, src, 64);
            group = g0 + src;
            first = glo + (int64_t)(tile - skipped) * TM;
            last = min(first + TM, ghi);
            return true;
        }
        before += __shfl(incl, 63, 64);
    }
    return false;
}

// silu(v) * up with silu(v) = v / (1 + exp(-v)), by the hardware's exp2 and reciprocal (within 2^-14 relative, far below
// bf16's half step of 2^-8). Far below zero, where exp(-v) leaves fp32's range and 1 + exp(v) is 1, silu(v) = v * exp(v)
// is taken as two factors, h = exp(v / 2) and v * h, and up goes between them: the result is right wherever h is a
// normal number (v >= -174), also where silu(v) alone would be none.
__device__ inline float silu_times(float v, float up) {
    const bool far = v < -40.0f;
    const float e = __builtin_amdgcn_exp2f(v * (far ? 0.72134752f : -1.44269504f));  // log2(e) / 2, -log2(e)
    const float f = far ? e : __builtin_amdgcn_rcpf(1.0f + e);
    return (v * f) * (far ? e * up : up);
}

__device__ inline __amdgpu_buffer_rsrc_t rsrc(const void *base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, (int32_t)min(bytes, (int64_t)0x7FFFFFFF),
                                             0x00020000);
}

// 16 bytes of each lane from the buffer at voff + soff straight to LDS, lane l's at dst + 16 l (dst the same for the
// whole wave); zero where the buffer ends before.
__device__ inline void load_to_lds(__amdgpu_buffer_rsrc_t src, uint8_t *dst, int voff, int soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void *)dst, 16, voff, soff, 0, 0);
}

// The groups' rows and tiles, in LDS: rows [lo, hi) of group g, and the number of row tiles up to its end.
struct TileTable {
    int32_t lo[MOE_MAX_EXPERTS], hi[MOE_MAX_EXPERTS], end[MOE_MAX_EXPERTS];
};

// One wave fills the table for row tiles of TM.
template <int TM>
__device__ inline void fill_table(TileTable &table, const int32_t *__restrict__ base, int G, int64_t a_rows) {
    const int lane = threadIdx.x & 63;
    int before = 0, reached = 0;
    for (int g0 = 0; g0 < G; g0 += 64) {
        const int g = g0 + lane;
        int lo, hi;
        group_rows(base, G, (int)a_rows, g0, reached, lo, hi);
        int incl = (hi - lo + TM - 1) / TM;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int u = __shfl_up(incl, d, 64);
            if (lane >= d) incl += u;
        }
        if (g < G) {
            table.lo[g] = lo;
            table.hi[g] = hi;
            table.end[g] = before + incl;
        }
        before += __shfl(incl, 63, 64);
    }
}

struct Tile {
    int group, first, rows, col;  // rows [first, first + rows) of the group, column tile col
};

// Tile t of the groups' row tiles x ncol column tiles, group by group, a group's row tiles fastest, so that
// the workgroups that an XCD runs at once share a few stretches of weights and rows in its L2.
template <int TM>
__device__ inline Tile find_tile(const TileTable &table, int G, int ncol, int t) {
    const int lane = threadIdx.x & 63;
    int g = 0;
    for (int g0 = 0; g0 < G; g0 += 64) {
        const uint64_t past = __ballot(g0 + lane < G && table.end[min(g0 + lane, G - 1)] * ncol <= t);
        g += __popcll(past);  // the groups that end before the tile come first
        if (past != ~0ull) break;
    }
    g = __builtin_amdgcn_readfirstlane(g);
    const int before = __builtin_amdgcn_readfirstlane(g > 0 ? table.end[g - 1] : 0);
    const int tiles = __builtin_amdgcn_readfirstlane(table.end[g]) - before;
    const int lo = __builtin_amdgcn_readfirstlane(table.lo[g]), hi = __builtin_amdgcn_readfirstlane(table.hi[g]);
    const int i = t - before * ncol, col = i / tiles, first = lo + (i - col * tiles) * TM;
    return Tile{g, first, min(TM, hi - first), col};
}

// Waits until at most N of the wave's loads are in flight and its LDS accesses are done, then for all waves.
template <int N>
__device__ inline void stage_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

}  // namespace product
}  // namespace moe
