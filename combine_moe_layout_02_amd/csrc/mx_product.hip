// The experts' product of MX E2M1 rows and weights for gfx950 (see moe_mx_product in moe.h).
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies a 16 x 128 by a 128 x 16 tile of E2M1 codes, lane l giving 32
// consecutive codes (16 bytes) of row l % 16, k-block l / 16, of either operand, and the E8M0 scale of
// exactly these 32: an MX block is a lane's operand. The weights are the first operand, so that a lane's
// four results are neighbouring outputs of one row.

#include "mx_blocks.h"

namespace moe {
namespace {

using namespace mx;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// One such product with byte S of the scale registers (operand formats 4 = E2M1).
template <int S>
__device__ inline f32x4 mfma_byte(const i32x4 &a, int a_scale, const i32x4 &b, int b_scale, const f32x4 &c) {
    const i32x8 a8 = {a.x, a.y, a.z, a.w, 0, 0, 0, 0}, b8 = {b.x, b.y, b.z, b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, S, a_scale, S, b_scale);
}

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

// The transpose of 4 x 4 bytes: word q of the result has byte q of the four words.
__device__ inline u32x4 transpose_bytes(const u32x4 &m) {
    const uint32_t lo01 = __builtin_amdgcn_perm(m[1], m[0], 0x05010400), hi01 = __builtin_amdgcn_perm(m[1], m[0], 0x07030602);
    const uint32_t lo23 = __builtin_amdgcn_perm(m[3], m[2], 0x05010400), hi23 = __builtin_amdgcn_perm(m[3], m[2], 0x07030602);
    return u32x4{__builtin_amdgcn_perm(lo23, lo01, 0x05040100), __builtin_amdgcn_perm(lo23, lo01, 0x07060302),
                 __builtin_amdgcn_perm(hi23, hi01, 0x05040100), __builtin_amdgcn_perm(hi23, hi01, 0x07060302)};
}

// Bytes `from` .. + 15 of a row of n, zero behind its end: loaded now, put in place later, so that nothing waits
// here. A row's last 16 bytes at the latest are loaded, and moved down when placed; SHORT rows (n < 16) go byte
// by byte.
template <bool SHORT>
__device__ inline u32x4 load_row16(const uint8_t *row, int from, int n) {
    u32x4 v = {0, 0, 0, 0};
    if constexpr (!SHORT) {
        __builtin_memcpy(&v, row + min(from, n - 16), 16);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (from + i < n) v[i >> 2] |= (uint32_t)row[from + i] << (8 * (i & 3));
    }
    return v;
}

template <bool SHORT>
__device__ inline u32x4 place_row16(const u32x4 &v, int from, int n) {
    if constexpr (SHORT) return v;
    const int down = max(from - (n - 16), 0);
    const unsigned __int128 wide = __builtin_bit_cast(unsigned __int128, v);
    return __builtin_bit_cast(u32x4, down == 0 ? wide : down >= 16 ? 0 : wide >> (8 * down));
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

// Tiles of TM rows x TN weight rows (TN / 2 outputs when GATED), WMC x WNC waves, through LDS. The 8 XCDs get
// contiguous eighths of the tiles (workgroup b runs on XCD b % 8).
//
// Codes go from memory straight to LDS in pairs of stages of 128 values, 128 bytes of a row (whole lines; stages
// of 64 bytes through a ring of four took 10% longer where the weights' bytes count), through PAIRS buffers: while
// one is multiplied the others fill. Scales come through registers, 16 blocks (four stages, one round) at a time, and
// lie in LDS so that one word holds a lane's four scales of a round. One barrier a pair: it follows each wave's wait
// for its own loads of the pair and for its LDS reads of the last one, so behind it the pair is whole and the last
// pair's buffer is free.
//
// PAIRS == 2, many tiles: a workgroup takes tile after tile, the next tile's first pair behind a tile's last, so that
// the loads never pause and a tile's results are stored while the next one's rows arrive.
//
// 32768 rows on 32 groups, 7168 -> 4096 gated, take 541 to 566 us in a stream of such calls (groups of uneven size; 504
// where every group fills its tiles), half of it with matrix instructions under way, and 570 to 650 in runs of 20 calls
// behind a pause. In a copy of the kernel with parts taken out, in such runs, where the whole took 636: the matrix cores alone 290 to 350 on random codes (the card's power
// holds them at 6.5 PFLOP/s), the loads alone 450, the products with their reads of LDS 500. Four waves of 128 x 128
// results read a third less of LDS, but took 700 there, and 718 with the next stage's operands read ahead: one wave a
// SIMD leaves its loads and reads uncovered.
//
// Row tiles are whole: one of a few rows takes the time of a full one and its weights again, so uneven groups whose mean
// fills the tiles cost more than even ones (7168 -> 4096 gated, uneven and even, us: 8 groups of 128 rows 41 and 33, 32
// of 128 149 and 125, of 256 203 and 153, of 512 336 and 266).
//
// PAIRS > 2, tiles for every compute unit once at most: a workgroup takes one tile, whose time is its pairs' way
// from memory and through the matrix cores: 0.55 us a pair with one under way and 0.45 with three at 64 x 128, 0.31
// at 64 x 64, 0.27 at 32 x 64 (with seven under way no less: there the reads and products of one wave count).
constexpr int kStageBlocks = 4;    // MX blocks of a stage
constexpr int kRoundStages = 4;    // stages of a round: two pairs
constexpr int kScaleBlocks = 16;   // MX blocks of a round

// Waits until at most N of the wave's loads are in flight and its LDS accesses are done, then for all waves.
template <int N>
__device__ inline void stage_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int TM, int TN, int WMC, int WNC, int PAIRS, bool GATED, bool SHORT>
__global__ __launch_bounds__(64 * WMC * WNC) void product_tile_kernel(
    const uint8_t *__restrict__ a_codes, const uint8_t *__restrict__ a_scales, int64_t a_rows,
    const int32_t *__restrict__ base, int G, const uint8_t *__restrict__ w_codes,
    const uint8_t *__restrict__ w_scales, int O, int nblk, int ncol, uint8_t *__restrict__ out,
    int64_t out_stride, bool wide) {
    constexpr int NW = WMC * WNC, THREADS = 64 * NW;
    constexpr int ROWS = TM + TN, WM = TM / WMC, WN = TN / WNC, MI = WM / 16, NI = WN / 16;
    constexpr int LOADS = ROWS / 8 / NW;                    // 8 rows of a pair of stages a load
    constexpr int SLOADS = (ROWS + THREADS - 1) / THREADS;  // rows of a round of scales a thread
    constexpr int OF = GATED ? NI / 2 : NI;                 // column fragments of results
    constexpr int STORES = MI * OF / 2;                     // stores of a wave, 16 bytes a lane
    static_assert((PAIRS == 2 || PAIRS == 4) && LOADS * 8 * NW == ROWS && OF % 2 == 0 && MI * 16 * WMC == TM && NI * 16 * WNC == TN, "shape");
    // the buffers are objects of their own, so that the compiler sees the reads of one and the loads into the
    // other apart and puts no wait between them
    __shared__ __align__(1024) uint8_t pair0[ROWS * 128], pair1[ROWS * 128];
    __shared__ __align__(1024) uint8_t pair2[PAIRS > 2 ? ROWS * 128 : 16], pair3[PAIRS > 2 ? ROWS * 128 : 16];
    uint8_t *const codes[4] = {pair0, pair1, pair2, pair3};
    __shared__ __align__(16) uint8_t scales[2][SLOADS * THREADS * 16];  // threads past the rows put the last one again
    __shared__ TileTable table;

    const int width = GATED ? O / 2 : O;
    const int pitch = nblk * 16;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (wave == 0) fill_table<TM>(table, base, G, a_rows);
    __syncthreads();
    const int all = __builtin_amdgcn_readfirstlane(table.end[G - 1]) * ncol, share = (all + 7) >> 3;
    const int xcd_end = min(((int)(blockIdx.x & 7) + 1) * share, all), step = gridDim.x >> 3;
    int t = (int)(blockIdx.x & 7) * share + (int)(blockIdx.x >> 3);
    if (t >= xcd_end) return;

    // Load l of a wave takes tile rows 8 (wave + l * NW) .. + 7, a lane 16 bytes: place lane % 8 of row lane / 8.
    // Place p of row r holds block p ^ (r % 8): eight neighbouring rows' reads of one block then cover all the
    // banks.
    const int r8 = lane >> 3, blk = (lane & 7) ^ r8;

    // What a thread loads of a tile: its rows' places in the codes and its row(s) of scales.
    struct Source {
        __amdgpu_buffer_rsrc_t a, w;
        int base[LOADS];  // byte offset of the load's first row, the same for the whole wave
        const uint8_t *scales[SLOADS];
    };
    const auto source_of = [&](const Tile &tile) {
        Source src;
        src.a = rsrc(a_codes + (int64_t)tile.first * pitch, (int64_t)tile.rows * pitch);
        src.w = rsrc(w_codes + (int64_t)tile.group * O * pitch, (int64_t)O * pitch);
        const int o0 = tile.col * (GATED ? TN / 2 : TN);
        // Row of the weights behind tile row j: plain, neighbours; gated, each wave's share of the tile has its
        // gate rows first, then the up rows of the same outputs. Rows past the matrix read as zero, rows past the
        // gates are up rows: neither's results are stored.
        const auto weight_row = [&](int j) {
            if (!GATED) return o0 + j;
            const int part = j / WN, jj = j % WN, o = o0 + part * (WN / 2) + jj % (WN / 2);
            return jj < WN / 2 ? o : width + o;
        };
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
            const int r = 8 * (wave + l * NW);
            src.base[l] = (r < TM ? r : weight_row(r - TM)) * pitch;
        }
#pragma unroll
        for (int l = 0; l < SLOADS; ++l) {
            const int r = min(l * THREADS + tid, ROWS - 1);
            src.scales[l] = r < TM ? a_scales + ((int64_t)tile.first + min(r, tile.rows - 1)) * nblk
                                   : w_scales + ((int64_t)tile.group * O + min(weight_row(r - TM), O - 1)) * nblk;
        }
        return src;
    };

    const int place = r8 * pitch + blk * 16;
    const auto load_codes = [&](const Source &src, int st, uint8_t *buf, bool none) {
        const bool past = none || st * kStageBlocks + blk >= nblk;  // blocks behind the row's end read as zero
#pragma unroll
        for (int l = 0; l < LOADS; ++l)
            load_to_lds(8 * (wave + l * NW) < TM ? src.a : src.w, &buf[(wave + l * NW) * 1024],
                        past ? 0x7FFFFFF0 : src.base[l] + place, st * 64);
    };
    u32x4 sreg[PAIRS / 2][SLOADS];  // rounds of the rows' scales, 16 bytes each
    const auto load_scales = [&](const Source &src, int round, u32x4 (&to)[SLOADS]) {
#pragma unroll
        for (int l = 0; l < SLOADS; ++l) to[l] = load_row16<SHORT>(src.scales[l], round * kScaleBlocks, nblk);
    };
    // Put as [row][lane's k-block q][stage of the round]: the transpose of the row's 4 x 4 bytes.
    const auto put_scales = [&](int round, int buf, const u32x4 (&from)[SLOADS]) {
#pragma unroll
        for (int l = 0; l < SLOADS; ++l)
            *reinterpret_cast<u32x4 *>(&scales[buf][(l * THREADS + tid) * 16]) =
                transpose_bytes(place_row16<SHORT>(from[l], round * kScaleBlocks, nblk));
    };

    const int wm = (wave % WMC) * WM, wn = TM + (wave / WMC) * WN;
    const int fr = lane & 15, q = lane >> 4;
    const int at0 = fr * 128 + (q ^ (fr & 7)) * 16, at1 = fr * 128 + ((q + 4) ^ (fr & 7)) * 16;
    const int stages = (nblk + kStageBlocks - 1) / kStageBlocks, rounds = (stages + kRoundStages - 1) / kRoundStages;

    f32x4 acc[MI][NI];
    int as[MI], ws[NI];
    i32x4 a[MI], w[NI];
    const auto read_scales = [&](int buf) {
#pragma unroll
        for (int j = 0; j < NI; ++j)
            ws[j] = *reinterpret_cast<const int *>(&scales[buf][(wn + j * 16 + fr) * 16 + q * 4]);
#pragma unroll
        for (int i = 0; i < MI; ++i)
            as[i] = *reinterpret_cast<const int *>(&scales[buf][(wm + i * 16 + fr) * 16 + q * 4]);
    };
    const auto read_codes = [&](const uint8_t *buf, int at) {
#pragma unroll
        for (int j = 0; j < NI; ++j) w[j] = *reinterpret_cast<const i32x4 *>(&buf[(wn + j * 16) * 128 + at]);
#pragma unroll
        for (int i = 0; i < MI; ++i) a[i] = *reinterpret_cast<const i32x4 *>(&buf[(wm + i * 16) * 128 + at]);
    };
    const auto multiply = [&](int s) {  // s: the stage's number in its round, a constant where this is unrolled
#pragma unroll
        for (int i = 0; i < MI; ++i) {
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                f32x4 &c = acc[i][j];
                if (s == 0) c = mfma_byte<0>(w[j], ws[j], a[i], as[i], c);
                else if (s == 1) c = mfma_byte<1>(w[j], ws[j], a[i], as[i], c);
                else if (s == 2) c = mfma_byte<2>(w[j], ws[j], a[i], as[i], c);
                else c = mfma_byte<3>(w[j], ws[j], a[i], as[i], c);
            }
        }
    };

    Tile tile = find_tile<TM>(table, G, ncol, t);
    Source cur = source_of(tile);
#pragma unroll
    for (int r = 0; r < PAIRS / 2; ++r) load_scales(cur, r, sreg[r]);
#pragma unroll
    for (int i = 0; i < PAIRS - 1; ++i) load_codes(cur, 2 * i, codes[i], false);
    int sbuf = 0;         // the scales' buffer of this round
    bool stored = false;  // the stores of the tile before are still in flight, STORES of them
    put_scales(0, 0, sreg[0]);
    for (;;) {
        t += step;
        const bool more = PAIRS == 2 && t < xcd_end;
        Tile next = tile;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
        if constexpr (PAIRS > 2) {
            // All but one of the pairs are under way while that one is multiplied; a round's scales are loaded as many
            // rounds ahead as the pairs are, so that the wait for them is none for codes that are not needed yet.
            for (int round = 0; round < rounds; round += PAIRS / 2) {
#pragma unroll
                for (int s = 0; s < 2 * PAIRS; ++s) {
                    const int st = round * kRoundStages + s, r = s / kRoundStages;
                    if (s % 2 == 0) stage_barrier<(PAIRS - 2) * LOADS>();
                    if (s % kRoundStages == 0) {
                        read_scales(r & 1);
                        load_scales(cur, round + r + PAIRS / 2, sreg[r]);
                    }
                    read_codes(codes[s >> 1], s & 1 ? at1 : at0);
                    if (s % 2 == 0) load_codes(cur, st + 2 * (PAIRS - 1), codes[((s >> 1) + PAIRS - 1) % PAIRS], false);
                    __builtin_amdgcn_sched_barrier(0);
                    if (st < stages) multiply(s % kRoundStages);
                    __builtin_amdgcn_sched_barrier(0);
                    if (s % kRoundStages == kRoundStages - 1)
                        put_scales(round + r + 1, (r + 1) & 1, sreg[(r + 1) % (PAIRS / 2)]);
                }
            }
        } else {
            for (int round = 0; round < rounds; ++round) {
                const bool last = round + 1 == rounds;
#pragma unroll
                for (int s = 0; s < kRoundStages; ++s) {
                    const int st = round * kRoundStages + s;
                    if ((s & 1) == 0) {
                        if (s == 0 && round == 0 && stored) stage_barrier<STORES>();
                        else stage_barrier<0>();
                    }
                    if (s == 0) read_scales(sbuf);
                    read_codes(codes[s >> 1], s & 1 ? at1 : at0);
                    if (s == 0) {
                        load_codes(cur, st + 2, codes[1], false);
                        if (last && more) {
                            next = find_tile<TM>(table, G, ncol, t);
                            cur = source_of(next);
                        }
                        load_scales(cur, last ? 0 : round + 1, sreg[0]);
                    }
                    // behind the tile's last pair comes the next tile's first one
                    if (s == 2) load_codes(cur, last ? 0 : st + 2, codes[0], last && !more);
                    __builtin_amdgcn_sched_barrier(0);  // the reads and loads are under way before the products
                    if (st < stages) multiply(s);
                    __builtin_amdgcn_sched_barrier(0);
                    if (s == kRoundStages - 1) {
                        sbuf ^= 1;
                        put_scales(last ? 0 : round + 1, sbuf, sreg[0]);
                    }
                }
            }
        }

        // A lane holds four neighbouring results of a row; swapping 16-lane rows between two column fragments
        // gives it eight, 16 bytes. With aligned rows every store goes out, past the tile's end to nowhere, so
        // that the next stages' waits know how many there are.
        const int o0 = tile.col * (GATED ? TN / 2 : TN) + (wave / WMC) * (GATED ? WN / 2 : WN);
        const __amdgpu_buffer_rsrc_t dst = rsrc(out + tile.first * out_stride, wide ? tile.rows * out_stride : 0);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int r = wm + i * 16 + fr;
#pragma unroll
            for (int j = 0; j < OF; j += 2) {
                uint32_t v[2][2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float f[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        f[e] = GATED ? silu_times(acc[i][j + k][e], acc[i][(j + k + OF) % NI][e]) : acc[i][j + k][e];
                    v[k][0] = bf16_pair(f[0], f[1]);
                    v[k][1] = bf16_pair(f[2], f[3]);
                }
                const auto lo = __builtin_amdgcn_permlane16_swap(v[0][0], v[1][0], false, false);
                const auto hi = __builtin_amdgcn_permlane16_swap(v[0][1], v[1][1], false, false);
                const u32x4 r8 = {lo[0], hi[0], lo[1], hi[1]};
                const int o = o0 + (j + (q & 1)) * 16 + (q >> 1) * 8;
                if (wide) {
                    const bool in = r < tile.rows && o < width;
                    __builtin_amdgcn_raw_buffer_store_b128(r8, dst, in ? r * (int)out_stride + o * 2 : 0x7FFFFFF0, 0, 0);
                } else if (r < tile.rows) {
                    uint16_t *to = reinterpret_cast<uint16_t *>(out + ((int64_t)tile.first + r) * out_stride) + o;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (o + e < width) to[e] = (uint16_t)(r8[e >> 1] >> (16 * (e & 1)));
                }
            }
        }
        stored = wide;
        if (!more) break;
        tile = next;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may reach LDS after the wave's end
}

// Few rows a group: the weights' bytes bound the product. A workgroup takes 16 rows of a group and 32 weight
// rows (16 outputs when GATED), its four waves a quarter of H each, and every wave streams its quarter
// through a ring of its own in LDS, waiting for nobody; the partial sums meet in LDS and are added in the
// waves' order. LDS turns the loads' order (four lanes to a row, 64 bytes) into the matrix cores' (a lane
// to a row): loaded straight to registers in their order, each lane's 16 bytes are an access of the L1 of
// their own, and 8 rows on 32 groups, H = 7168, O = 4096, took 32 us.
constexpr int kSmallWaves = 4;
constexpr int kRing = 4;  // buffers of a wave's ring, of 128 values each

template <bool GATED, bool SHORT>
__global__ __launch_bounds__(64 * kSmallWaves) void product_small_kernel(
    const uint8_t *__restrict__ a_codes, const uint8_t *__restrict__ a_scales, int64_t a_rows,
    const int32_t *__restrict__ base, int G, const uint8_t *__restrict__ w_codes,
    const uint8_t *__restrict__ w_scales, int O, int nblk, uint8_t *__restrict__ out, int64_t out_stride) {
    constexpr int F = 3, ROWS = 16 * F;  // fragments of 16 rows: the rows, then two of the weights
    __shared__ __align__(1024) uint8_t ring0[kSmallWaves][F * 1024], ring1[kSmallWaves][F * 1024], ring2[kSmallWaves][F * 1024],
        ring3[kSmallWaves][F * 1024];
    __shared__ __align__(16) uint8_t scales[kSmallWaves][64 * 16];  // a lane puts a row, the last lanes one again
    int g;
    int64_t first, last;
    const int col = blockIdx.y;
    if (!find_rows<16>(base, G, a_rows, blockIdx.x, g, first, last)) return;
    g = __builtin_amdgcn_readfirstlane(g);
    first = __builtin_amdgcn_readfirstlane((int)first);
    last = __builtin_amdgcn_readfirstlane((int)last);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, q = lane >> 4;
    const int width = GATED ? O / 2 : O, o0 = col * (GATED ? 16 : 32), pitch = nblk * 16;
    uint8_t *const codes[kRing] = {ring0[wave], ring1[wave], ring2[wave], ring3[wave]};
    const int rows = (int)(last - first);
    const __amdgpu_buffer_rsrc_t a_src = rsrc(a_codes + first * pitch, (int64_t)rows * pitch);
    const __amdgpu_buffer_rsrc_t w_src = rsrc(w_codes + (int64_t)g * O * pitch, (int64_t)O * pitch);
    // row r of the tile's ROWS, in its own matrix; rows past the end repeat the last one
    const auto row_of = [&](int r) {
        if (r < 16) return min(r, rows - 1);
        const int j = r - 16;
        return GATED ? min(o0 + (j & 15), width - 1) + (j >> 4) * width : min(o0 + j, width - 1);
    };
    const int r4 = lane >> 2, blk = (lane & 3) ^ ((r4 >> 1) & 3);  // places against bank conflicts, as in the tiles
    int voff[F];
#pragma unroll
    for (int f = 0; f < F; ++f) voff[f] = row_of(16 * f + r4) * pitch + blk * 16;

    const int steps = (nblk + kStageBlocks - 1) / kStageBlocks;
    const int share = (steps + kSmallWaves - 1) / kSmallWaves;
    const int begin = min(wave * share, steps), count = min(share, steps - begin);
    const auto load_codes = [&](int i, uint8_t *buf) {  // step i of the wave's
        const bool past = i >= count || (begin + i) * kStageBlocks + blk >= nblk;
#pragma unroll
        for (int f = 0; f < F; ++f)
            load_to_lds(f == 0 ? a_src : w_src, &buf[f * 1024], past ? 0x7FFFFFF0 : voff[f], (begin + i) * 64);
    };
    const int srow_at = min(lane, ROWS - 1);
    const uint8_t *srow = srow_at < 16 ? a_scales + (first + row_of(srow_at)) * nblk
                                       : w_scales + ((int64_t)g * O + row_of(srow_at)) * nblk;

    f32x4 acc[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
    u32x4 sreg = load_row16<SHORT>(srow, begin * kStageBlocks, nblk);
#pragma unroll
    for (int s = 0; s < kRing - 1; ++s) load_codes(s, codes[s]);
    const int at = fr * 64 + (q ^ ((fr >> 1) & 3)) * 16;
    const auto put_scales = [&](int i0) {
        *reinterpret_cast<u32x4 *>(&scales[wave][lane * 16]) =
            transpose_bytes(place_row16<SHORT>(sreg, (begin + i0) * kStageBlocks, nblk));
    };
    put_scales(0);
    for (int i0 = 0; i0 < count; i0 += kRing) {
        int sc[F];  // a lane's scales of this round's four steps, one word a fragment
#pragma unroll
        for (int f = 0; f < F; ++f) sc[f] = *reinterpret_cast<const int *>(&scales[wave][(f * 16 + fr) * 16 + q * 4]);
        sreg = load_row16<SHORT>(srow, (begin + i0 + kRing) * kStageBlocks, nblk);
#pragma unroll
        for (int s = 0; s < kRing; ++s) {
            __builtin_amdgcn_sched_barrier(0);  // the scales' load stays above, their use below
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((kRing - 2) * F) : "memory");
            load_codes(i0 + s + kRing - 1, codes[(s + kRing - 1) % kRing]);
            i32x4 v[F];
#pragma unroll
            for (int f = 0; f < F; ++f) v[f] = *reinterpret_cast<const i32x4 *>(&codes[s][f * 1024 + at]);
            if (i0 + s < count) {  // behind them the codes are zero, but a scale may be a NaN
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    f32x4 &c = acc[j];
                    if (s == 0) c = mfma_byte<0>(v[1 + j], sc[1 + j], v[0], sc[0], c);
                    else if (s == 1) c = mfma_byte<1>(v[1 + j], sc[1 + j], v[0], sc[0], c);
                    else if (s == 2) c = mfma_byte<2>(v[1 + j], sc[1 + j], v[0], sc[0], c);
                    else c = mfma_byte<3>(v[1 + j], sc[1 + j], v[0], sc[0], c);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            if (s == kRing - 1) put_scales(i0 + kRing);
        }
    }
    // every load has arrived before the rings hold sums, and before the wave ends
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();
    f32x4 *const partial = reinterpret_cast<f32x4 *>(&ring0[0][0]);  // [wave][fragment][lane]
#pragma unroll
    for (int j = 0; j < 2; ++j) partial[(wave * 2 + j) * 64 + lane] = acc[j];
    __syncthreads();
    // the first wave adds and stores gate and up, the first two a fragment each of a plain product
    if (wave >= (GATED ? 1 : 2)) return;
    f32x4 sum = {0, 0, 0, 0}, up = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < kSmallWaves; ++k) {
        sum += partial[(k * 2 + wave) * 64 + lane];
        if (GATED) up += partial[(k * 2 + 1) * 64 + lane];
    }
    if (fr >= rows) return;
    uint16_t *dst = reinterpret_cast<uint16_t *>(out + (first + fr) * out_stride);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int o = o0 + 16 * wave + 4 * q + e;
        if (o < width) dst[o] = (uint16_t)bf16_pair(GATED ? silu_times(sum[e], up[e]) : sum[e], 0.0f);
    }
}

hipError_t few_rows(const void *a_codes, const void *a_scales, int64_t a_rows, const int32_t *group_base,
                    int32_t G, const void *w_codes, const void *w_scales, int32_t O, int32_t H, bool gated,
                    void *out, int64_t out_stride, hipStream_t stream) {
    const int64_t row_tiles = a_rows / 16 + (a_rows < G ? a_rows : G);  // at most
    const int ncol = gated ? (O / 2 + 15) / 16 : (O + 31) / 32;
    auto *kernel = H >= 512 ? (gated ? product_small_kernel<true, false> : product_small_kernel<false, false>)
                            : (gated ? product_small_kernel<true, true> : product_small_kernel<false, true>);
    hipLaunchKernelGGL(kernel, dim3((uint32_t)row_tiles, ncol), dim3(64 * kSmallWaves), 0, stream,
                       static_cast<const uint8_t *>(a_codes), static_cast<const uint8_t *>(a_scales), a_rows,
                       group_base, G, static_cast<const uint8_t *>(w_codes),
                       static_cast<const uint8_t *>(w_scales), O, H / 32, static_cast<uint8_t *>(out), out_stride);
    return hipGetLastError();
}

constexpr int kUnits = 256;  // compute units of an MI355X

// MIN_H: the least H that the caller's rule has for this tile; rows of scales below 16 bytes (H < 512) have their kernel
// only where it can come to them.
template <int TM, int TN, int WMC, int WNC, int PAIRS, int MIN_H = 32>
hipError_t tiles(const void *a_codes, const void *a_scales, int64_t a_rows, const int32_t *group_base,
                 int32_t G, const void *w_codes, const void *w_scales, int32_t O, int32_t H, bool gated,
                 void *out, int64_t out_stride, bool wide, hipStream_t stream) {
    constexpr int resident = TM + TN > 256 ? kUnits : 2 * kUnits;  // workgroups that run at once, by their LDS
    const int width = gated ? O / 2 : O, tn = gated ? TN / 2 : TN;
    const int ncol = (width + tn - 1) / tn;
    const int64_t row_tiles = a_rows / TM + (a_rows < G ? a_rows : G);  // at most
    const int64_t need = (row_tiles * ncol + 7) / 8 * 8;
    const int64_t grid = PAIRS > 2 || need < resident ? need : resident;
    auto *kernel = gated ? product_tile_kernel<TM, TN, WMC, WNC, PAIRS, true, false>
                         : product_tile_kernel<TM, TN, WMC, WNC, PAIRS, false, false>;
    if constexpr (MIN_H < 512) {
        if (H < 512)
            kernel = gated ? product_tile_kernel<TM, TN, WMC, WNC, PAIRS, true, true>
                           : product_tile_kernel<TM, TN, WMC, WNC, PAIRS, false, true>;
    }
    hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(64 * WMC * WNC), 0, stream,
                       static_cast<const uint8_t *>(a_codes), static_cast<const uint8_t *>(a_scales),
                       a_rows, group_base, G, static_cast<const uint8_t *>(w_codes),
                       static_cast<const uint8_t *>(w_scales), O, H / 32, ncol,
                       static_cast<uint8_t *>(out), out_stride, wide);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_product(const void *a_codes, const void *a_scales, int64_t a_rows,
                             const int32_t *group_base, int32_t G, const void *w_codes,
                             const void *w_scales, int32_t O, int32_t H, int32_t epilogue, void *out,
                             int64_t out_stride_bytes, hipStream_t stream) {
    if (a_rows == 0) return hipSuccess;
    const bool gated = epilogue == MOE_MX_GATED;
    const int width = gated ? O / 2 : O;
    // rows of whole 16-byte pieces, and a tile of them within a buffer descriptor's range
    const bool wide = width % 8 == 0 && out_stride_bytes % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0 &&
                      out_stride_bytes <= (1 << 22);
    // Which kernel, by the tiles it would have if the rows were spread over as many groups as they can reach, a
    // quarter of them more in the fuller ones. One run over the kernels, weights from memory, uneven groups (us; groups x
    // rows a group):
    //   7168 -> 4096 gated   1x8    1x64   1x256  1x512  4x16   4x32   8x32   8x64   4x128  8x128  32x16  32x64  32x256
    //   few_rows             6.9    17.6                 32.2   36.5   68.7                        221
    //   32 x 64, four pairs  11.6   11.9   15.8   28.6   16.8   23.9   45.1   58.4   48.7   82.7   100    198    536
    //   64 x 64, four        13.1   13.1   14.5   21.4   17.1   18.2   31.2   41.3   35.7   57.7   102    157    404
    //   64 x 128, four       16.9   17.3   17.8   20.2   22.2   23.7   28.1   45.1   41.4   63.3   98.0   141    383
    //   128 x 128, four             23.0   23.9   26.2          26.2   30.3   31.8   29.1   55.5          139    325
    //   64 x 128, two        19.4   19.9   20.3   22.4   30.1   30.3   33.5   43.1   38.5   63.5   91.4   130    323
    //   128 x 128, two              23.2   23.9   25.4          32.5   35.6   36.1   33.8   50.7          108    255
    //   256 x 256, two              47.8   48.8   50.0                        58.2   58.0   61.4          146    234
    // and 2048 -> 7168, 1x64, in the same order: 11.3, 6.4, 6.7, 8.1, 10.2, 8.6, 9.8, 17.7.
    // Where the tiles are no more than the compute units, all of a tile's time is its way through one, and small
    // tiles with more pairs under way shorten it; few_rows, whose waves share H, is ahead while its workgroups read
    // no more than 15360 rows (5x101, 6528 -> 220: 8.3 against 11.8). Four pairs of a large tile leave room for one
    // workgroup a compute unit, which short rows do not repay (1024 -> 1024 gated, 32x32: 64 x 128 8.2 against 7.5;
    // 32x64: 128 x 128 9.9 against 8.7). With more tiles the two pairs' kernels, which start a tile while they end
    // another, are ahead, the larger the more rows there are to share the weights: 128 x 128 from 300 tiles (16
    // groups, 3001 rows, 1056 -> 1000, 256 tiles: 12.4 against 10.2), 256 x 256 where they fill the compute units
    // (2048 -> 7168, 8x256, 448 tiles: 44.1 against 40.3; 32x256: 135 against 139).
    const int64_t hit = a_rows < G ? a_rows : G, mean = (a_rows + hit - 1) / hit;
    const int64_t most = hit > 1 ? mean + mean / 4 : mean;
    const auto tiles_of = [&](int tm, int tn) {
        const int outs = gated ? tn / 2 : tn;
        return hit * ((most + tm - 1) / tm) * ((width + outs - 1) / outs);
    };
    if (tiles_of(16, 32) * ((most < 16 ? most : 16) + 32) <= 320 * 48)  // rows that its workgroups read
        return few_rows(a_codes, a_scales, a_rows, group_base, G, w_codes, w_scales, O, H, gated, out,
                        out_stride_bytes, stream);
    if (tiles_of(32, 64) <= (most <= 32 ? 448 : kUnits))  // two at once on a compute unit, and room for a fuller group
        return tiles<32, 64, 2, 1, 4>(a_codes, a_scales, a_rows, group_base, G, w_codes, w_scales, O, H, gated, out,
                                      out_stride_bytes, wide, stream);
    if (tiles_of(64, 64) <= kUnits)
        return tiles<64, 64, 4, 1, 4>(a_codes, a_scales, a_rows, group_base, G, w_codes, w_scales, O, H, gated, out,
                                      out_stride_bytes, wide, stream);
    if (H >= 2048 && tiles_of(64, 128) <= kUnits)
        return tiles<64, 128, 2, 2, 4, 2048>(a_codes, a_scales, a_rows, group_base, G, w_codes, w_scales, O, H, gated, out,
                                             out_stride_bytes, wide, stream);
    if (H >= 4096 && tiles_of(128, 128) <= kUnits)
        return tiles<128, 128, 2, 2, 4, 4096>(a_codes, a_scales, a_rows, group_base, G, w_codes, w_scales, O, H, gated, out,
                                              out_stride_bytes, wide, stream);
    const int64_t large = tiles_of(256, 256);
    if (mean >= 160 && (large >= 4 * kUnits || (H >= 4096 && large >= 192 && large <= kUnits)))
        return tiles<256, 256, 2, 4, 2>(a_codes, a_scales, a_rows, group_base, G, w_codes, w_scales, O, H, gated, out,
                                        out_stride_bytes, wide, stream);
    if (mean >= 40 && tiles_of(128, 128) >= 300)
        return tiles<128, 128, 2, 2, 2>(a_codes, a_scales, a_rows, group_base, G, w_codes, w_scales, O, H, gated, out,
                                        out_stride_bytes, wide, stream);
    return tiles<64, 128, 2, 2, 2>(a_codes, a_scales, a_rows, group_base, G, w_codes, w_scales, O, H, gated, out,
                                   out_stride_bytes, wide, stream);
}

}  // namespace moe
