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

__device__ inline f32x4 mfma(const i32x4 &a, int a_scale, const i32x4 &b, int b_scale, const f32x4 &c) {
    const i32x8 a8 = {a.x, a.y, a.z, a.w, 0, 0, 0, 0}, b8 = {b.x, b.y, b.z, b.w, 0, 0, 0, 0};
    // operand formats 4 = E2M1; the scale is the low byte of its register
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, 0, a_scale, 0, b_scale);
}

// The same with byte S of the scale registers.
template <int S>
__device__ inline f32x4 mfma_byte(const i32x4 &a, int a_scale, const i32x4 &b, int b_scale, const f32x4 &c) {
    const i32x8 a8 = {a.x, a.y, a.z, a.w, 0, 0, 0, 0}, b8 = {b.x, b.y, b.z, b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, S, a_scale, S, b_scale);
}

// The rows [first, last) that tile number `tile` covers, TM rows at most, and their group; false when there
// are fewer tiles. Groups' tiles follow one another; every lane of a wave calls this and gets the same.
template <int TM>
__device__ inline bool find_tile(const int32_t *__restrict__ base, int G, int64_t a_rows, int tile,
                                 int &group, int64_t &first, int64_t &last) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int g0 = 0; g0 < G; g0 += 64) {
        const int g = g0 + lane;
        int64_t lo = 0, hi = 0;
        if (g < G) {
            lo = min(max((int64_t)base[g], (int64_t)0), a_rows);
            hi = min(max((int64_t)base[g + 1], lo), a_rows);
        }
        const int tiles = (int)((hi - lo + TM - 1) / TM);
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
            const int64_t glo = __shfl((int)lo, src, 64), ghi = __shfl((int)hi, src, 64);
            group = g0 + src;
            first = glo + (int64_t)(tile - skipped) * TM;
            last = min(first + TM, ghi);
            return true;
        }
        before += __shfl(incl, 63, 64);
    }
    return false;
}

__device__ inline float silu(float v) { return v / (1.0f + __expf(-v)); }

__device__ inline __amdgpu_buffer_rsrc_t rsrc(const void *base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, (int32_t)min(bytes, (int64_t)0x7FFFFFFF),
                                             0x00020000);
}

// 16 bytes of each lane from the buffer at voff + soff straight to LDS, lane l's at dst + 16 l (dst the same for the
// whole wave); zero where the buffer ends before.
__device__ inline void load_to_lds(__amdgpu_buffer_rsrc_t src, uint8_t *dst, int voff, int soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void *)dst, 16, voff, soff, 0, 0);
}

// Four neighbouring results of one row: columns o .. o + 3 of [0, width).
__device__ inline void store4(uint8_t *row, int o, int width, bool wide, const float (&v)[4]) {
    const uint32_t lo = bf16_pair(v[0], v[1]), hi = bf16_pair(v[2], v[3]);
    uint16_t *dst = reinterpret_cast<uint16_t *>(row) + o;
    if (wide && o + 4 <= width) {
        *reinterpret_cast<u32x2 *>(dst) = u32x2{lo, hi};
        return;
    }
    if (o < width) dst[0] = (uint16_t)lo;
    if (o + 1 < width) dst[1] = (uint16_t)(lo >> 16);
    if (o + 2 < width) dst[2] = (uint16_t)hi;
    if (o + 3 < width) dst[3] = (uint16_t)(hi >> 16);
}

// The tile that workgroup b of the grid takes, of all row tiles x column tiles: the 8 XCDs get contiguous
// eighths of the tiles (workgroup b runs on XCD b % 8), group by group, row tiles of a group fastest, so
// that the workgroups running at once on an XCD share a few stretches of weights and rows in its L2.
template <int TM>
__device__ inline bool find_tile(const int32_t *__restrict__ base, int G, int64_t a_rows, int ncol, int &group,
                                 int64_t &first, int64_t &last, int &col) {
    const int lane = threadIdx.x & 63;
    int total = 0;
    for (int g0 = 0; g0 < G; g0 += 64) {
        int tiles = 0;
        if (g0 + lane < G) {
            const int64_t lo = min(max((int64_t)base[g0 + lane], (int64_t)0), a_rows);
            const int64_t hi = min(max((int64_t)base[g0 + lane + 1], lo), a_rows);
            tiles = (int)((hi - lo + TM - 1) / TM);
        }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) tiles += __shfl_xor(tiles, d, 64);
        total += tiles;
    }
    const int64_t all = (int64_t)total * ncol, share = (all + 7) >> 3;
    const int64_t i = blockIdx.x >> 3;
    int64_t t = (blockIdx.x & 7) * share + i;
    if (i >= share || t >= all) return false;
    int64_t before = 0;
    for (int g0 = 0; g0 < G; g0 += 64) {
        int64_t lo = 0, hi = 0;
        if (g0 + lane < G) {
            lo = min(max((int64_t)base[g0 + lane], (int64_t)0), a_rows);
            hi = min(max((int64_t)base[g0 + lane + 1], lo), a_rows);
        }
        const int tiles = (int)((hi - lo + TM - 1) / TM);
        int incl = tiles;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int u = __shfl_up(incl, d, 64);
            if (lane >= d) incl += u;
        }
        const uint64_t here = __ballot(t < (before + incl) * ncol);
        if (here) {
            const int src = __ffsll((unsigned long long)here) - 1;
            const int rows = __shfl(tiles, src, 64);
            const int64_t in_group = t - (before + __shfl(incl - tiles, src, 64)) * ncol;
            const int64_t glo = __shfl((int)lo, src, 64), ghi = __shfl((int)hi, src, 64);
            group = __builtin_amdgcn_readfirstlane(g0 + src);
            col = __builtin_amdgcn_readfirstlane((int)(in_group / rows));
            first = __builtin_amdgcn_readfirstlane((int)(glo + (in_group % rows) * TM));
            last = min(first + TM, (int64_t)__builtin_amdgcn_readfirstlane((int)ghi));
            return true;
        }
        before += __shfl(incl, 63, 64);
    }
    return false;
}

// Tiles of TM rows x TN weight rows (TN / 2 outputs when GATED), WMC x WNC waves, through LDS.
//
// Codes go from memory straight to LDS in stages of 128 values (64 bytes of a row) through a ring of four
// buffers, and from there to registers one stage ahead of the products: while the matrix cores work on stage
// s, its successor is read from LDS and stage s + 4 is loaded into the buffer that stage s has left. Scales
// come through registers, 16 blocks (four stages, one round) at a time, and lie in LDS so that one word holds
// a lane's four scales of a round. One barrier a stage: it follows each wave's wait for its own loads of the
// next stage and for its LDS reads of this one, so behind it the next stage is whole and this buffer is free.
constexpr int kRing = 4;
constexpr int kStageBlocks = 4;    // MX blocks of a stage
constexpr int kScaleBlocks = 16;   // MX blocks of a round of scales: kRing stages

// Waits until at most N of the wave's loads are in flight and its LDS accesses are done, then for all waves.
template <int N>
__device__ inline void stage_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int TM, int TN, int WMC, int WNC, bool GATED>
__global__ __launch_bounds__(64 * WMC * WNC) void product_tile_kernel(
    const uint8_t *__restrict__ a_codes, const uint8_t *__restrict__ a_scales, int64_t a_rows,
    const int32_t *__restrict__ base, int G, const uint8_t *__restrict__ w_codes,
    const uint8_t *__restrict__ w_scales, int O, int nblk, int ncol, uint8_t *__restrict__ out,
    int64_t out_stride, bool wide) {
    constexpr int NW = WMC * WNC, THREADS = 64 * NW;
    constexpr int ROWS = TM + TN, WM = TM / WMC, WN = TN / WNC, MI = WM / 16, NI = WN / 16;
    constexpr int LOADS = ROWS / 16 / NW;     // 16 rows of a stage a load
    constexpr int SLOADS = ROWS / THREADS;    // rows of a round of scales a thread
    static_assert(LOADS * 16 * NW == ROWS && SLOADS * THREADS == ROWS && kRing == 4, "shape");
    // the ring's buffers are objects of their own, so that the compiler sees a buffer's reads and another's
    // loads apart and puts no wait between them
    __shared__ __align__(1024) uint8_t ring0[ROWS * 64], ring1[ROWS * 64], ring2[ROWS * 64], ring3[ROWS * 64];
    uint8_t *const codes[kRing] = {ring0, ring1, ring2, ring3};
    __shared__ __align__(16) uint8_t scales[2][ROWS * 16];

    int g, col;
    int64_t first, last;
    if (!find_tile<TM>(base, G, a_rows, ncol, g, first, last, col)) return;
    g = __builtin_amdgcn_readfirstlane(g);
    col = __builtin_amdgcn_readfirstlane(col);
    first = __builtin_amdgcn_readfirstlane((int)first);
    last = __builtin_amdgcn_readfirstlane((int)last);
    const int width = GATED ? O / 2 : O;
    const int o0 = col * (GATED ? TN / 2 : TN);
    const int rows = (int)(last - first);
    const int pitch = nblk * 16;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const __amdgpu_buffer_rsrc_t a_src = rsrc(a_codes + first * pitch, (int64_t)rows * pitch);
    const __amdgpu_buffer_rsrc_t w_src = rsrc(w_codes + (int64_t)g * O * pitch, (int64_t)O * pitch);

    // Row of the weights behind tile row j: plain, neighbours; gated, each wave's share of the tile has its gate
    // rows first, then the up rows of the same outputs. Rows past the end repeat the last one.
    const auto weight_row = [&](int j) {
        if (!GATED) return min(o0 + j, width - 1);
        const int share = j / WN, jj = j % WN;
        const int o = min(o0 + share * (WN / 2) + jj % (WN / 2), width - 1);
        return jj < WN / 2 ? o : width + o;
    };

    // Load l of a wave takes tile rows 16 (wave + l * NW) .. + 15, a lane 16 bytes: place lane % 4 of row lane / 4.
    // Place p of row r holds block p ^ (r / 2 % 4): eight neighbouring rows' reads of one block then cover all
    // the banks (SQ_LDS_BANK_CONFLICT is 0).
    const int r4 = lane >> 2, blk = (lane & 3) ^ ((r4 >> 1) & 3);
    int voff[LOADS];
#pragma unroll
    for (int l = 0; l < LOADS; ++l) {
        const int r = 16 * (wave + l * NW) + r4;
        voff[l] = (r < TM ? min(r, rows - 1) : weight_row(r - TM)) * pitch + blk * 16;
    }
    const uint8_t *ssrc[SLOADS];
#pragma unroll
    for (int l = 0; l < SLOADS; ++l) {
        const int r = l * THREADS + tid;
        ssrc[l] = r < TM ? a_scales + (first + min(r, rows - 1)) * nblk
                         : w_scales + ((int64_t)g * O + weight_row(r - TM)) * nblk;
    }

    const auto load_codes = [&](int st, int buf) {
        const bool past = st * kStageBlocks + blk >= nblk;  // blocks behind the row's end read as zero
#pragma unroll
        for (int l = 0; l < LOADS; ++l)
            load_to_lds(16 * (wave + l * NW) < TM ? a_src : w_src, &codes[buf][(wave + l * NW) * 1024],
                        past ? 0x7FFFFFF0 : voff[l], st * 64);
    };
    u32x4 sreg[SLOADS];
    // A round of a row's scales: 16 bytes. Rounds that end behind the row take its last 16 bytes (nblk >= 16) and
    // are moved down when put, so that blocks behind the end have scale byte 0.
    const auto load_scales = [&](int round) {
        const int from = min(round * kScaleBlocks, nblk - kScaleBlocks);
#pragma unroll
        for (int l = 0; l < SLOADS; ++l) __builtin_memcpy(&sreg[l], ssrc[l] + from, 16);
    };
    // Put as [row][lane's k-block q][stage of the round]: the transpose of the row's 4 x 4 bytes.
    const auto put_scales = [&](int round, int buf) {
        const int down = min(max(round * kScaleBlocks - (nblk - kScaleBlocks), 0), 16);
#pragma unroll
        for (int l = 0; l < SLOADS; ++l) {
            const unsigned __int128 v = __builtin_bit_cast(unsigned __int128, sreg[l]);
            const unsigned __int128 moved = down == 0 ? v : down == 16 ? 0 : v >> (8 * down);
            const u32x4 m = __builtin_bit_cast(u32x4, moved);
            const uint32_t lo01 = __builtin_amdgcn_perm(m[1], m[0], 0x05010400), hi01 = __builtin_amdgcn_perm(m[1], m[0], 0x07030602);
            const uint32_t lo23 = __builtin_amdgcn_perm(m[3], m[2], 0x05010400), hi23 = __builtin_amdgcn_perm(m[3], m[2], 0x07030602);
            *reinterpret_cast<u32x4 *>(&scales[buf][(l * THREADS + tid) * 16]) =
                u32x4{__builtin_amdgcn_perm(lo23, lo01, 0x05040100), __builtin_amdgcn_perm(lo23, lo01, 0x07060302),
                      __builtin_amdgcn_perm(hi23, hi01, 0x05040100), __builtin_amdgcn_perm(hi23, hi01, 0x07060302)};
        }
    };

    f32x4 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    const int wm = (wave % WMC) * WM, wn = TM + (wave / WMC) * WN;
    const int fr = lane & 15, q = lane >> 4;
    const int at = fr * 64 + (q ^ ((fr >> 1) & 3)) * 16;

    i32x4 a[MI], w[NI];
    int as[MI], ws[NI];
    const auto read_codes = [&](const uint8_t *buf) {
#pragma unroll
        for (int j = 0; j < NI; ++j) w[j] = *reinterpret_cast<const i32x4 *>(&buf[(wn + j * 16) * 64 + at]);
#pragma unroll
        for (int i = 0; i < MI; ++i) a[i] = *reinterpret_cast<const i32x4 *>(&buf[(wm + i * 16) * 64 + at]);
    };
    const auto read_scales = [&](int buf) {
#pragma unroll
        for (int j = 0; j < NI; ++j) ws[j] = *reinterpret_cast<const int *>(&scales[buf][(wn + j * 16 + fr) * 16 + q * 4]);
#pragma unroll
        for (int i = 0; i < MI; ++i) as[i] = *reinterpret_cast<const int *>(&scales[buf][(wm + i * 16 + fr) * 16 + q * 4]);
    };

    const int stages = (nblk + kStageBlocks - 1) / kStageBlocks;
    load_scales(0);
#pragma unroll
    for (int s = 0; s < kRing - 1; ++s) load_codes(s, s);
    put_scales(0, 0);
    for (int round = 0; round * kRing < stages; ++round) {
#pragma unroll
        for (int s = 0; s < kRing; ++s) {
            const int st = round * kRing + s;
            if (st >= stages) break;
            stage_barrier<(kRing - 2) * LOADS>();
            if (s == 0) read_scales(round & 1);
            read_codes(codes[s]);
            if (s == 0) load_scales(round + 1);
            load_codes(st + kRing - 1, (s + kRing - 1) % kRing);
            __builtin_amdgcn_sched_barrier(0);  // the reads and loads are under way before the products
#pragma unroll
            for (int i = 0; i < MI; ++i) {
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    f32x4 &c = acc[i][j];
                    const i32x4 &x = a[i], &y = w[j];
                    if (s == 0) c = mfma_byte<0>(y, ws[j], x, as[i], c);
                    else if (s == 1) c = mfma_byte<1>(y, ws[j], x, as[i], c);
                    else if (s == 2) c = mfma_byte<2>(y, ws[j], x, as[i], c);
                    else c = mfma_byte<3>(y, ws[j], x, as[i], c);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            if (s == kRing - 1) put_scales(round + 1, (round + 1) & 1);
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may reach LDS after the wave's end

#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int r = wm + i * 16 + fr;
        if (r >= rows) continue;
        uint8_t *dst = out + (first + r) * out_stride;
#pragma unroll
        for (int j = 0; j < (GATED ? NI / 2 : NI); ++j) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = GATED ? silu(acc[i][j][e]) * acc[i][(j + NI / 2) % NI][e] : acc[i][j][e];
            store4(dst, o0 + (wave / WMC) * (GATED ? WN / 2 : WN) + j * 16 + 4 * q, width, wide, v);
        }
    }
}

// grid = (row tiles of 16, tiles of 16 outputs), one wave each, straight from memory.
template <bool GATED>
__global__ __launch_bounds__(64) void product_kernel(
    const uint8_t *__restrict__ a_codes, const uint8_t *__restrict__ a_scales, int64_t a_rows,
    const int32_t *__restrict__ base, int G, const uint8_t *__restrict__ w_codes,
    const uint8_t *__restrict__ w_scales, int O, int H, uint8_t *__restrict__ out,
    int64_t out_stride) {
    int g;
    int64_t first, last;
    if (!find_tile<16>(base, G, a_rows, blockIdx.x, g, first, last)) return;
    const int lane = threadIdx.x, r = lane & 15, q = lane >> 4;
    const int nblk = H / 32, width = GATED ? O / 2 : O;
    const int o0 = blockIdx.y * 16;
    const int64_t row = min(first + r, last - 1);          // lanes past the tile repeat its last row
    const int64_t wrow = (int64_t)g * O + min(o0 + r, width - 1);
    const int64_t urow = wrow + width;
    f32x4 acc = {0, 0, 0, 0}, up = {0, 0, 0, 0};
    for (int b0 = 0; b0 < nblk; b0 += 4) {
        const int b = b0 + q;
        const bool in = b < nblk;
        i32x4 x = {0, 0, 0, 0}, w = {0, 0, 0, 0}, u = {0, 0, 0, 0};
        int xs = 0, ws = 0, us = 0;
        if (in) {
            x = *reinterpret_cast<const i32x4 *>(a_codes + (row * nblk + b) * 16);
            xs = a_scales[row * nblk + b];
            w = *reinterpret_cast<const i32x4 *>(w_codes + (wrow * nblk + b) * 16);
            ws = w_scales[wrow * nblk + b];
            if (GATED) {
                u = *reinterpret_cast<const i32x4 *>(w_codes + (urow * nblk + b) * 16);
                us = w_scales[urow * nblk + b];
            }
        }
        acc = mfma(w, ws, x, xs, acc);
        if (GATED) up = mfma(u, us, x, xs, up);
    }
    if (first + r >= last) return;
    uint16_t *dst = reinterpret_cast<uint16_t *>(out + (first + r) * out_stride);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int o = o0 + 4 * q + i;
        if (o < width) dst[o] = (uint16_t)bf16_pair(GATED ? silu(acc[i]) * up[i] : acc[i], 0.0f);
    }
}

template <int TM, int TN, int WMC, int WNC>
hipError_t tiles(const void *a_codes, const void *a_scales, int64_t a_rows, const int32_t *group_base,
                 int32_t G, const void *w_codes, const void *w_scales, int32_t O, int32_t H, bool gated,
                 void *out, int64_t out_stride, bool wide, hipStream_t stream) {
    const int width = gated ? O / 2 : O, tn = gated ? TN / 2 : TN;
    const int ncol = (width + tn - 1) / tn;
    const int64_t row_tiles = a_rows / TM + (a_rows < G ? a_rows : G);  // at most
    const int64_t grid = (row_tiles * ncol + 7) / 8 * 8;
    auto *kernel = gated ? product_tile_kernel<TM, TN, WMC, WNC, true> : product_tile_kernel<TM, TN, WMC, WNC, false>;
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
    const int64_t row_tiles = a_rows / 16 + (a_rows < G ? a_rows : G);
    const bool wide = out_stride_bytes % 8 == 0 && reinterpret_cast<uintptr_t>(out) % 8 == 0;
    const int64_t mean = a_rows / G;
    if (mean >= 192 && H >= 512)
        return tiles<256, 256, 2, 4>(a_codes, a_scales, a_rows, group_base, G, w_codes, w_scales, O, H, gated, out,
                               out_stride_bytes, wide, stream);
    if (mean >= 32 && H >= 512)
        return tiles<128, 128, 2, 2>(a_codes, a_scales, a_rows, group_base, G, w_codes, w_scales, O, H, gated, out,
                               out_stride_bytes, wide, stream);
    auto *kernel = gated ? product_kernel<true> : product_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)row_tiles, (width + 15) / 16), dim3(64), 0, stream,
                       static_cast<const uint8_t *>(a_codes), static_cast<const uint8_t *>(a_scales),
                       a_rows, group_base, G, static_cast<const uint8_t *>(w_codes),
                       static_cast<const uint8_t *>(w_scales), O, H, static_cast<uint8_t *>(out),
                       out_stride_bytes);
    return hipGetLastError();
}

}  // namespace moe
