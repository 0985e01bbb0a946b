// The experts' product of INT8 rows and weights for gfx950 (see moe_scaled_product in moe.h).
//
// v_mfma_i32_16x16x64_i8 multiplies a 16 x 64 by a 64 x 16 tile, lane l giving 16 consecutive values (16 bytes) of row
// l % 16, k-block l / 16, of either operand. The weights are the first operand, so that a lane's four results are
// neighbouring outputs of one row. Sums are whole numbers below 2^31 (H * 128 * 128 <= 2^28), the same in any order.

#include <algorithm>

#include "product_rows.h"

namespace moe {
namespace {

using namespace product;

typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ inline i32x4 mfma(const i32x4 &a, const i32x4 &b, const i32x4 &c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// fp32(fp32(c * a) * w): a result's value from its sum and its two scales.
__device__ inline float scaled(int c, float a, float w) { return (float)c * a * w; }

// As find_tile, but a group's rows are shared evenly among its tiles, in steps of STEP, so that they take the same time, in
// step with one another over the weights they share; and of a tile's rows the piece-th of `pieces` shares. 32768 rows on 32 uneven
// groups, 7168 -> 4096 gated: 963 us with whole tiles and a rest, 925 like this.
template <int TM, int STEP>
__device__ inline Tile find_even_tile(const TileTable &table, int G, int ncol, int t, int piece, int pieces) {
    Tile tile = find_tile<TM>(table, G, ncol, t);
    const int lo = __builtin_amdgcn_readfirstlane(table.lo[tile.group]), hi = __builtin_amdgcn_readfirstlane(table.hi[tile.group]);
    const int n = hi - lo, tiles = (n + TM - 1) / TM;
    const int height = ((n + tiles - 1) / tiles + STEP - 1) / STEP * STEP;  // (tiles - 1) * height <= (tiles - 1) * TM < n
    const int first = lo + (tile.first - lo) / TM * height, rows = min(height, hi - first);
    const int part = ((rows + pieces - 1) / pieces + STEP - 1) / STEP * STEP;
    tile.first = first + piece * part;
    tile.rows = max(min(part, rows - piece * part), 0);  // less, or none, where the shares before have taken all
    return tile;
}

// Which tiles a workgroup takes: of its XCD's, begin .. end, every step-th from its own on; of a last round that would leave
// workgroups without one, each tile in as many pieces as there are workgroups for it.
struct Turns {
    int end, step, whole, mine;  // rounds that are whole, and the workgroup's number in its XCD
    int t, piece, pieces;

    __device__ Turns(int all, int most) {
        const int share = (all + 7) >> 3, begin = min((int)(blockIdx.x & 7) * share, all);
        end = min(begin + share, all);
        step = gridDim.x >> 3;
        mine = blockIdx.x >> 3;
        whole = begin + (end - begin) / step * step;
        t = begin + mine - step;
        piece = 0;
        pieces = 1;
        left = end - whole;
        split = left > 0 ? min(step / left, most) : 1;
    }
    // The next turn; false when there is none.
    __device__ bool next() {
        if (t + step < whole) {
            t += step;
            return true;
        }
        if (t >= whole || mine >= left * split) return false;
        t = whole + mine % left;
        piece = mine / left;
        pieces = split;
        return true;
    }
    int left, split;
};

// Tiles of TM rows x TN weight rows (TN / 2 outputs when GATED), WMC x WNC waves, through LDS. The 8 XCDs get
// contiguous eighths of the tiles (workgroup b runs on XCD b % 8).
//
// Codes go from memory straight to LDS in pairs of stages of 64 values, 128 bytes of a row (whole lines), through PAIRS
// buffers: while one is multiplied the others fill. One barrier a pair: it follows each wave's wait for its own loads of
// the pair and for its LDS reads of the last one, so behind it the pair is whole and the last pair's buffer is free.
//
// PAIRS == 2, many tiles: a workgroup takes tile after tile, the next tile's first pair behind a tile's last, so that
// the loads never pause and a tile's results are stored while the next one's rows arrive. 32768 rows on 32 even groups, 7168 -> 4096
// gated, take 820 to 870 us (2.2 to 2.35 PFLOP/s), uneven ones 910 to 950, with matrix instructions under way for 53% of the cycles
// at 2.18 GHz and no bank conflict. In copies of the kernel with parts taken out (even groups, 835 whole): the matrix
// instructions alone 548 (507 on zeros: the card's power), with the reads of LDS 632, the loads alone 700, all of it on
// rows that stay in an XCD's L2 762, on zeros 754. Not faster: the lines of later pairs brought to L2 ahead (the loads alone
// 568, the whole the same), loads before the reads, a fragment's second stage read while the first is multiplied, 32 x 32 x 32
// matrix instructions (1075), tiles of 320 x 256 (923, uneven 980), 256 x 128 and 128 x 256 (1041, 1076).
//
// Where the weights' bytes bound it (1024 rows on 32 groups, 2048 -> 7168: 90 us), a bare read of them in this pattern takes 74 and the
// results' stores 8 to 11; three pairs under way, strips of 64 to 256 weight rows, a first pair that differs from tile to
// tile, and a last round shared out by outputs took the same or longer.
//
// PAIRS > 2, tiles for every compute unit once at most: a workgroup takes one tile, whose time is its pairs' way
// from memory and through the matrix cores, 0.7 us a pair at 128 x 128.
template <int TM, int TN, int WMC, int WNC, int PAIRS, bool GATED>
__global__ __launch_bounds__(64 * WMC * WNC) void int8_tile_kernel(
    const uint8_t *__restrict__ a_codes, const float *__restrict__ a_scales, int64_t a_rows,
    const int32_t *__restrict__ base, int G, const uint8_t *__restrict__ w_codes,
    const float *__restrict__ w_scales, int O, int H, int ncol, uint8_t *__restrict__ out, int64_t out_stride,
    bool wide, bool lines) {
    constexpr int NW = WMC * WNC;
    constexpr int ROWS = TM + TN, WM = TM / WMC, WN = TN / WNC, MI = WM / 16, NI = WN / 16;
    constexpr int LOADS = ROWS / 8 / NW;     // 8 rows of a pair of stages a load
    constexpr int OF = GATED ? NI / 2 : NI;  // column fragments of results
    constexpr int STORES = MI * OF / 2;      // stores of a wave, 16 bytes a lane
    // Tiles of few rows, whose weights stream past, store whole lines with sc1 nt (decode batch, 1024 rows of 2048 -> 7168 on 32
    // groups: 89.4 us, and 93.4 written back; with the rows to 8 bits behind it 96.3 and 97.5). Parts of lines are
    // joined in the caches (3001 rows, 1040 -> 1000: 12.0 us, and 14.6 with sc1 nt), and large tiles' results stay there for
    // the call that reads them (8192 rows as above 174.8 and 174.7, with the call behind 204.5 and 206.9).
    constexpr bool STREAMS = TM < 256;
    static_assert((PAIRS == 2 || PAIRS == 4) && LOADS * 8 * NW == ROWS && OF % 2 == 0 && MI * 16 * WMC == TM && NI * 16 * WNC == TN, "shape");
    // the buffers are objects of their own, so that the compiler sees the reads of one and the loads into the
    // other apart and puts no wait between them
    __shared__ __align__(1024) uint8_t pair0[ROWS * 128], pair1[ROWS * 128];
    __shared__ __align__(1024) uint8_t pair2[PAIRS > 2 ? ROWS * 128 : 16], pair3[PAIRS > 2 ? ROWS * 128 : 16];
    uint8_t *const codes[4] = {pair0, pair1, pair2, pair3};
    __shared__ TileTable table;

    const int width = GATED ? O / 2 : O;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (wave == 0) fill_table<TM>(table, base, G, a_rows);
    __syncthreads();
    Turns turn(__builtin_amdgcn_readfirstlane(table.end[G - 1]) * ncol, PAIRS == 2 ? TM / (16 * WMC) : 1);
    if (!turn.next()) return;

    // Load l of a wave takes tile rows 8 (wave + l * NW) .. + 7, a lane 16 bytes: place lane % 8 of row lane / 8.
    // Place p of row r holds block p ^ (r % 8): eight neighbouring rows' reads of one block then cover all the
    // banks.
    const int r8 = lane >> 3, blk = (lane & 7) ^ r8;
    struct Source {
        __amdgpu_buffer_rsrc_t a, w;
        int base[LOADS];  // byte offset of the load's first row, the same for the whole wave
    };
    const auto source_of = [&](const Tile &tile) {
        Source src;
        src.a = rsrc(a_codes + (int64_t)tile.first * H, (int64_t)tile.rows * H);
        src.w = rsrc(w_codes + (int64_t)tile.group * O * H, (int64_t)O * H);
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
            src.base[l] = (r < TM ? r : weight_row(r - TM)) * H;
        }
        return src;
    };
    const int place = r8 * H + blk * 16;
    const auto load_codes = [&](const Source &src, int pair, uint8_t *buf, bool none) {
        const bool past = none || pair * 128 + blk * 16 >= H;  // blocks behind the row's end read as zero
#pragma unroll
        for (int l = 0; l < LOADS; ++l)
            load_to_lds(8 * (wave + l * NW) < TM ? src.a : src.w, &buf[(wave + l * NW) * 1024],
                        past ? 0x7FFFFFF0 : src.base[l] + place, pair * 128);
    };

    const int wn = TM + (wave / WMC) * WN;
    const int fr = lane & 15, q = lane >> 4;
    const int at0 = fr * 128 + (q ^ (fr & 7)) * 16, at1 = fr * 128 + ((q + 4) ^ (fr & 7)) * 16;
    const int stages = (H + 63) / 64, pairs = (stages + 1) / 2;

    i32x4 acc[MI][NI];
    i32x4 a[MI], w[NI];
    // The waves share a tile's rows evenly, mi fragments each: a constant number of them, or (most 0) whatever mi is, whose
    // tests take 7% longer.
    int mi, wm;
    const auto taken = [&](auto most, int i) { return most.value > 0 ? i < most.value : i < mi; };
    const auto read_codes = [&](auto most, const uint8_t *buf, int at) {
#pragma unroll
        for (int j = 0; j < NI; ++j) w[j] = *reinterpret_cast<const i32x4 *>(&buf[(wn + j * 16) * 128 + at]);
#pragma unroll
        for (int i = 0; i < MI; ++i)
            if (taken(most, i)) a[i] = *reinterpret_cast<const i32x4 *>(&buf[(wm + i * 16) * 128 + at]);
    };
    const auto multiply = [&](auto most) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
            if (taken(most, i)) {
#pragma unroll
                for (int j = 0; j < NI; ++j) acc[i][j] = mfma(w[j], a[i], acc[i][j]);
            }
    };

    const auto tile_of = [&]() { return find_even_tile<TM, 16 * WMC>(table, G, ncol, turn.t, turn.piece, turn.pieces); };
    Tile tile = tile_of();
    Source cur = source_of(tile);
#pragma unroll
    for (int i = 0; i < PAIRS - 1; ++i) load_codes(cur, i, codes[i], false);
    bool stored = false;  // the stores of the tile before are still in flight, STORES of them
    for (;;) {
        const bool more = PAIRS == 2 && turn.next();
        Tile next = tile;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
        mi = (tile.rows + 16 * WMC - 1) / (16 * WMC);
        wm = (wave % WMC) * mi * 16;
        // a round is a pair in each buffer, so that a buffer's number is a constant
        const auto all_rounds = [&](auto most) {
            for (int p0 = 0; p0 < pairs; p0 += PAIRS) {
                const bool last = p0 + PAIRS >= pairs;
#pragma unroll
                for (int b = 0; b < PAIRS; ++b) {
                    const int p = p0 + b;
                    if (PAIRS == 2 && b == 0 && p0 == 0 && stored) stage_barrier<STORES>();
                    else stage_barrier<(PAIRS - 2) * LOADS>();
                    read_codes(most, codes[b], at0);
                    if (PAIRS > 2) {
                        load_codes(cur, p + PAIRS - 1, codes[(b + PAIRS - 1) % PAIRS], false);
                    } else if (b == 0) {
                        load_codes(cur, p + 1, codes[1], false);
                        if (last && more) {
                            next = tile_of();
                            cur = source_of(next);
                        }
                    } else {
                        // behind the tile's last pair comes the next tile's first one
                        load_codes(cur, last ? 0 : p + 1, codes[0], last && !more);
                    }
                    __builtin_amdgcn_sched_barrier(0);  // the reads and loads are under way before the products
                    if (p < pairs) multiply(most);
                    __builtin_amdgcn_sched_barrier(0);
                    read_codes(most, codes[b], at1);
                    if (2 * p + 1 < stages) multiply(most);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        };
        if (mi == MI) all_rounds(std::integral_constant<int, MI>{});
        else if (MI > 1 && mi == MI - 1) all_rounds(std::integral_constant<int, MI - 1>{});
        else if (MI > 2 && mi == MI - 2) all_rounds(std::integral_constant<int, MI - 2>{});
        else if (MI > 3) all_rounds(std::integral_constant<int, 0>{});

        // A lane holds four neighbouring results of a row; swapping 16-lane rows between two column fragments
        // gives it eight, 16 bytes. With aligned rows every store goes out, past the tile's end to nowhere, so
        // that the next stages' waits know how many there are.
        const int o0 = tile.col * (GATED ? TN / 2 : TN) + (wave / WMC) * (GATED ? WN / 2 : WN);
        const __amdgpu_buffer_rsrc_t dst = rsrc(out + tile.first * out_stride, wide ? tile.rows * out_stride : 0);
        const __amdgpu_buffer_rsrc_t sa_src = rsrc(a_scales + tile.first, tile.rows * 4);
        const __amdgpu_buffer_rsrc_t sw_src = rsrc(w_scales + (int64_t)tile.group * O, (int64_t)O * 4);
        float sa[MI];
        float sw[NI][4];
#pragma unroll
        for (int i = 0; i < MI; ++i)
            sa[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(sa_src, (wm + i * 16 + fr) * 4, 0, 0));
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sw[j][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                    sw_src, (o0 + (j % OF) * 16 + 4 * q + e + (j >= OF ? width : 0)) * 4, 0, 0));
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
                    for (int e = 0; e < 4; ++e) {
                        const int up = (j + k + OF) % NI;
                        f[e] = scaled(acc[i][j + k][e], sa[i], sw[j + k][e]);
                        if (GATED) f[e] = silu_times(f[e], scaled(acc[i][up][e], sa[i], sw[up][e]));
                    }
                    v[k][0] = bf16_pair(f[0], f[1]);
                    v[k][1] = bf16_pair(f[2], f[3]);
                }
                const auto lo = __builtin_amdgcn_permlane16_swap(v[0][0], v[1][0], false, false);
                const auto hi = __builtin_amdgcn_permlane16_swap(v[0][1], v[1][1], false, false);
                const u32x4 r8 = {lo[0], hi[0], lo[1], hi[1]};
                const int o = o0 + (j + (q & 1)) * 16 + (q >> 1) * 8;
                if (wide) {
                    const bool in = i < mi && r < tile.rows && o < width;
                    const int at = in ? r * (int)out_stride + o * 2 : 0x7FFFFFF0;
                    if (STREAMS && lines) __builtin_amdgcn_raw_buffer_store_b128(r8, dst, at, 0, 16 | 2);
                    else __builtin_amdgcn_raw_buffer_store_b128(r8, dst, at, 0, 0);
                } else if (i < mi && r < tile.rows) {
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

// Few rows a group: the weights' bytes bound the product, and the way of a wave's share of H (8 rows on one group, 7168 -> 4096
// gated: 13.2 us; with eight waves 14.2, with two 14.2). A workgroup takes 16 rows of a group and 32 weight
// rows (16 outputs when GATED), its four waves a quarter of H each, and every wave streams its quarter
// through a ring of its own in LDS, waiting for nobody; the partial sums meet in LDS. LDS turns the loads' order (four
// lanes to a row, 64 bytes) into the matrix cores' (a lane to a row).
constexpr int kSmallWaves = 4;
constexpr int kRing = 4;  // buffers of a wave's ring, of 64 values each

template <bool GATED>
__global__ __launch_bounds__(64 * kSmallWaves) void int8_small_kernel(
    const uint8_t *__restrict__ a_codes, const float *__restrict__ a_scales, int64_t a_rows,
    const int32_t *__restrict__ base, int G, const uint8_t *__restrict__ w_codes,
    const float *__restrict__ w_scales, int O, int H, uint8_t *__restrict__ out, int64_t out_stride) {
    constexpr int F = 3;  // fragments of 16 rows: the rows, then two of the weights
    __shared__ __align__(1024) uint8_t ring0[kSmallWaves][F * 1024], ring1[kSmallWaves][F * 1024], ring2[kSmallWaves][F * 1024],
        ring3[kSmallWaves][F * 1024];
    int g;
    int64_t first, last;
    const int col = blockIdx.y;
    if (!find_rows<16>(base, G, a_rows, blockIdx.x, g, first, last)) return;
    g = __builtin_amdgcn_readfirstlane(g);
    first = __builtin_amdgcn_readfirstlane((int)first);
    last = __builtin_amdgcn_readfirstlane((int)last);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, q = lane >> 4;
    const int width = GATED ? O / 2 : O, o0 = col * (GATED ? 16 : 32);
    uint8_t *const codes[kRing] = {ring0[wave], ring1[wave], ring2[wave], ring3[wave]};
    const int rows = (int)(last - first);
    const __amdgpu_buffer_rsrc_t a_src = rsrc(a_codes + first * H, (int64_t)rows * H);
    const __amdgpu_buffer_rsrc_t w_src = rsrc(w_codes + (int64_t)g * O * H, (int64_t)O * H);
    // row r of the tile's, in its own matrix; rows past the end repeat the last one
    const auto row_of = [&](int r) {
        if (r < 16) return min(r, rows - 1);
        const int j = r - 16;
        return GATED ? min(o0 + (j & 15), width - 1) + (j >> 4) * width : min(o0 + j, width - 1);
    };
    const int r4 = lane >> 2, blk = (lane & 3) ^ ((r4 >> 1) & 3);  // places against bank conflicts, as in the tiles
    int voff[F];
#pragma unroll
    for (int f = 0; f < F; ++f) voff[f] = row_of(16 * f + r4) * H + blk * 16;

    const int steps = (H + 63) / 64;
    const int share = (steps + kSmallWaves - 1) / kSmallWaves;
    const int begin = min(wave * share, steps), count = min(share, steps - begin);
    const auto load_codes = [&](int i, uint8_t *buf) {  // step i of the wave's
        const bool past = i >= count || (begin + i) * 64 + blk * 16 >= H;
#pragma unroll
        for (int f = 0; f < F; ++f)
            load_to_lds(f == 0 ? a_src : w_src, &buf[f * 1024], past ? 0x7FFFFFF0 : voff[f], (begin + i) * 64);
    };
    i32x4 acc[2] = {i32x4{0, 0, 0, 0}, i32x4{0, 0, 0, 0}};
#pragma unroll
    for (int s = 0; s < kRing - 1; ++s) load_codes(s, codes[s]);
    const int at = fr * 64 + (q ^ ((fr >> 1) & 3)) * 16;
    for (int i0 = 0; i0 < count; i0 += kRing) {
#pragma unroll
        for (int s = 0; s < kRing; ++s) {
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((kRing - 2) * F) : "memory");
            load_codes(i0 + s + kRing - 1, codes[(s + kRing - 1) % kRing]);
            i32x4 v[F];
#pragma unroll
            for (int f = 0; f < F; ++f) v[f] = *reinterpret_cast<const i32x4 *>(&codes[s][f * 1024 + at]);
            // behind the wave's steps the codes are zero
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[j] = mfma(v[1 + j], v[0], acc[j]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // every load has arrived before the rings hold sums, and before the wave ends
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();
    i32x4 *const partial = reinterpret_cast<i32x4 *>(&ring0[0][0]);  // [wave][fragment][lane]
#pragma unroll
    for (int j = 0; j < 2; ++j) partial[(wave * 2 + j) * 64 + lane] = acc[j];
    __syncthreads();
    // the first wave adds and stores gate and up, the first two a fragment each of a plain product
    if (wave >= (GATED ? 1 : 2)) return;
    i32x4 sum = {0, 0, 0, 0}, up = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < kSmallWaves; ++k) {
        sum += partial[(k * 2 + wave) * 64 + lane];
        if (GATED) up += partial[(k * 2 + 1) * 64 + lane];
    }
    if (fr >= rows) return;
    const float sa = a_scales[first + fr];
    const float *sw = w_scales + (int64_t)g * O;
    uint16_t *dst = reinterpret_cast<uint16_t *>(out + (first + fr) * out_stride);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int o = o0 + 16 * wave + 4 * q + e;
        if (o >= width) continue;
        float v = scaled(sum[e], sa, sw[o]);
        if (GATED) v = silu_times(v, scaled(up[e], sa, sw[width + o]));
        dst[o] = (uint16_t)bf16_pair(v, 0.0f);
    }
}

struct Args {
    const uint8_t *a_codes;
    const float *a_scales;
    int64_t a_rows;
    const int32_t *base;
    int G;
    const uint8_t *w_codes;
    const float *w_scales;
    int O, H;
    bool gated;
    uint8_t *out;
    int64_t out_stride;
    bool wide, lines;
    hipStream_t stream;
};

hipError_t few_rows(const Args &p) {
    const int64_t row_tiles = p.a_rows / 16 + (p.a_rows < p.G ? p.a_rows : p.G);  // at most
    const int ncol = p.gated ? (p.O / 2 + 15) / 16 : (p.O + 31) / 32;
    auto *kernel = p.gated ? int8_small_kernel<true> : int8_small_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)row_tiles, ncol), dim3(64 * kSmallWaves), 0, p.stream, p.a_codes,
                       p.a_scales, p.a_rows, p.base, p.G, p.w_codes, p.w_scales, p.O, p.H, p.out, p.out_stride);
    return hipGetLastError();
}

constexpr int kUnits = 256;  // compute units of an MI355X

template <int TM, int TN, int WMC, int WNC, int PAIRS>
hipError_t tiles(const Args &p) {
    constexpr int resident = (TM + TN) * PAIRS > 640 ? kUnits : 2 * kUnits;  // workgroups that run at once, by their LDS
    const int width = p.gated ? p.O / 2 : p.O, tn = p.gated ? TN / 2 : TN;
    const int ncol = (width + tn - 1) / tn;
    const int64_t row_tiles = p.a_rows / TM + (p.a_rows < p.G ? p.a_rows : p.G);  // at most
    const int64_t need = (row_tiles * ncol + 7) / 8 * 8;
    const int64_t grid = PAIRS > 2 || need < resident ? need : resident;
    auto *kernel = p.gated ? int8_tile_kernel<TM, TN, WMC, WNC, PAIRS, true> : int8_tile_kernel<TM, TN, WMC, WNC, PAIRS, false>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(64 * WMC * WNC), 0, p.stream, p.a_codes, p.a_scales, p.a_rows,
                       p.base, p.G, p.w_codes, p.w_scales, p.O, p.H, ncol, p.out, p.out_stride, p.wide, p.lines);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_product(const void *a_codes, const float *a_scales, int64_t a_rows,
                               const int32_t *group_base, int32_t G, const void *w_codes,
                               const float *w_scales, int32_t O, int32_t H, int32_t epilogue,
                               void *out, int64_t out_stride_bytes, hipStream_t stream) {
    if (a_rows == 0) return hipSuccess;
    const bool gated = epilogue == MOE_MX_GATED;
    const int width = gated ? O / 2 : O;
    // rows of whole 16-byte pieces, and a tile of them within a buffer descriptor's range
    const bool wide = width % 8 == 0 && out_stride_bytes % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0 &&
                      out_stride_bytes <= (1 << 22);
    const bool lines = wide && out_stride_bytes % 128 == 0 && reinterpret_cast<uintptr_t>(out) % 128 == 0;
    const Args p = {static_cast<const uint8_t *>(a_codes), a_scales, a_rows, group_base, G,
                    static_cast<const uint8_t *>(w_codes), w_scales, O, H, gated, static_cast<uint8_t *>(out),
                    out_stride_bytes, wide, lines, stream};
    // Which kernel, by the tiles it would have if the rows were spread over as many groups as they can reach, a quarter of
    // them more in the fuller ones. One run over the kernels, weights from memory, uneven groups (us; groups x rows a group):
    //   7168 -> 4096 gated   1x8    1x64   1x256  1x512  1x2000*  4x16   4x32   4x128  8x32   8x64   8x128  32x2   32x16  32x64  32x256
    //   few_rows             13.2   27.3                          48.2
    //   32 x 64, four pairs  18.2   18.6   26.1                   23.7   32.2          63.2                 144    162
    //   64 x 64, four        18.9   21.3   20.9   33.0   68.5     23.8   25.0   51.5   47.0   61.9   90.1   138    160    222    517
    //   64 x 128, four       24.4   30.2   29.3   29.7   52.7     29.9   32.7   58.1   44.3   64.2   87.1   146    162    200    480
    //   128 x 128, four      27.8   32.0   39.2   39.8   40.6     32.3   34.4   42.9   44.9   49.8   79.9                 184    393
    //   64 x 128, two                      48.1   48.5   55.6                   57.3   57.9   64.1   103    142    159    195    461
    //   128 x 128, two                            54.1   55.0                   58.3          62.9   73.9   150    163    182    349
    //   256 x 256, two                                                                               97.7                 203    313
    // (* 2048 outputs), and others, in the same order from 64 x 128 with four:
    //   rows a group         1x12288  1x3000  4x512  8x200   8x256  16x188  20x300  40x63  50x240  64x313  1x32768
    //   H -> outputs         1024 1024 2048 4096 1024 4096 4096 4096g 2048 7168 1040 1000 3008 512g 2048 2048g 800 640 512 512 256 128
    //   64 x 128, four       43.9     59.4             68.8            20.5    35.8    48.4
    //   128 x 128, four      35.3     45.7    30.5     60.7    70.8    15.9    25.9    47.0   33.1    24.9    9.2
    //   64 x 128, two        32.5     52.1    28.2     65.4    70.3    16.1    30.7    42.5   30.6    21.0    7.6
    //   128 x 128, two       30.2     42.4    25.7     58.3    62.1    16.3    32.9    48.3   27.6    19.6    8.1
    //   256 x 256, two       24.1     35.2    23.1     61.1    59.9                           24.8    18.4    11.3
    // Where the tiles are no more than the compute units, all of a tile's time is its way through one, and small tiles
    // with more pairs under way shorten it; few_rows, whose waves share H, is ahead while its workgroups read no more
    // than 12288 rows. Its steps of 64 bytes of a row are half lines, or parts of two, which costs it where they come
    // from memory: 291 rows on 19 groups, 6400 -> 222, 11.9 and 16.3 with 32 x 64; 134 on 30, 6256 -> 300, 26.5 and
    // 19.0, 86 on one, 6560 -> 1134 (7 MB of weights), 12.1 and 16.6. With more tiles the two pairs' kernels, which
    // start a tile while they end another, are ahead, the larger the more rows there are to share the weights: 128 x 128
    // from 48 rows a group and, for short rows, 300 tiles (15766 rows on 32 groups, 7104 -> 148 gated, 278 of them: 71
    // and 90 with 64 x 128), 256 x 256 from 160 rows and 192 tiles (its last round goes out in pieces). But up to 24
    // rows a group 64 x 64 with four pairs gets the bytes sooner, as its rounds are shorter: 85 rows on 32 groups, 6032
    // -> 2192 gated, 85.9 and 121 with 64 x 128 and two, 1019 on 61, 5488 -> 1074 gated, 86.8 and 113, 512 on 32, 7168
    // -> 4096 gated, 161 and 158.
    //
    // 256 x 256 also wants its columns filled. One column of 128 weight rows leaves half of every tile without results: 65536
    // rows on 8 groups, 256 -> 128 gated, 21.2 and 11.7 with 128 x 128, 2^20 rows on one, 4096 -> 128, 1034 and 915. Three
    // columns leave a quarter, which long rows make up for and short ones do not: 65536 rows on 8 groups, 256 -> 384, 27.1
    // and 20.5, 262144 on one, 4096 -> 384, 508 and 645. Over 310 products of 49152 to 2^20 rows on 1 or 8 groups, 256 to
    // 4096 -> 64 to 1000, the choice takes 1.6% longer than the best of the two pairs' kernels, 37% at most; without
    // this condition 9.3% and 81%.
    //
    // Four pairs want rows of 12 pairs: 3001 rows on 16 groups, 1040 -> 1000, take 15.9 with 128 x 128 and four, 16.1
    // with 64 x 128 and two from memory, 15.4 and 12.0 from the caches; 43 rows on 64 groups, 1520 -> 3494 gated, 38.5
    // with 64 x 64 and four, 38.4.
    //
    // How many tiles uneven groups have is expected, from their mean: a half more than their rows would fill, one at
    // least. Over 514 products of random sizes (1 to 32768 rows on 1 to 64 groups, 4 MB of weights at least) the rule's
    // choice takes 1.7% longer than the best of these kernels (geometric mean); with each group's tiles counted at five
    // quarters of the mean it took 5.7. Over 450 others, of up to 2^20 rows on up to 512 groups, it is 1.8% behind, 42% at most
    // (290 rows on 6 groups, 7104 -> 2229), and a bound of 1024, 1280, 2048 or 2560 on H in place of 1536 makes it 1.9, 1.8, 1.8
    // and 1.9.
    const int64_t hit = a_rows < G ? a_rows : G, mean = (a_rows + hit - 1) / hit;
    const auto expected = [&](int tm, int tn) {
        const int outs = gated ? tn / 2 : tn;
        const int64_t halves = hit > 1 ? std::max<int64_t>(2 * tm, 2 * mean + tm) : (mean + tm - 1) / tm * 2 * tm;  // of tm rows a group, times tm
        return hit * ((width + outs - 1) / outs) * halves / (2 * tm);
    };
    const int64_t reads = expected(16, 32) * (std::min<int64_t>(mean, 16) + 32);  // rows that few_rows' workgroups read
    const int cols = gated ? 64 : 128, columns = (width + cols - 1) / cols, spare = columns % 2;  // of 128 weight rows, one alone in a tile of 256
    const bool filled = spare * 5 <= columns || (H >= 1536 && spare * 3 <= columns);
    const bool cached = hit * O * H <= 12 << 20 || reads * H <= 56 << 20;
    if (reads <= 12288 && (H % 64 == 0 || cached)) return few_rows(p);
    if (expected(32, 64) <= (mean <= 32 ? 2 * kUnits : kUnits)) return tiles<32, 64, 2, 1, 4>(p);  // two at once on a unit
    if (expected(64, 64) <= kUnits) return tiles<64, 64, 4, 1, 4>(p);
    if (expected(64, 128) <= kUnits) return tiles<64, 128, 2, 2, 4>(p);
    if (mean <= 24 && H >= 1536) return tiles<64, 64, 4, 1, 4>(p);
    if (mean >= 160 && filled && expected(256, 256) >= 192) return tiles<256, 256, 2, 4, 2>(p);
    if (H >= 1536 && expected(128, 128) <= kUnits) return tiles<128, 128, 2, 2, 4>(p);
    if (mean >= 48 && (H >= 1536 || expected(128, 128) >= 300)) return tiles<128, 128, 2, 2, 2>(p);
    return tiles<64, 128, 2, 2, 2>(p);
}

}  // namespace moe
