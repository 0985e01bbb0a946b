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

constexpr int kTileThreads = 256;
constexpr int kStageBlocks = 8;   // MX blocks of a stage: 256 values, 128 bytes of a row

// A tile of TM rows x TN weight rows (TN / 2 outputs when GATED), four waves as 2 x 2, K in stages of 256.
template <int TM, int TN, bool GATED>
__global__ __launch_bounds__(kTileThreads) void product_tile_kernel(
    const uint8_t *__restrict__ a_codes, const uint8_t *__restrict__ a_scales, int64_t a_rows,
    const int32_t *__restrict__ base, int G, const uint8_t *__restrict__ w_codes,
    const uint8_t *__restrict__ w_scales, int O, int nblk, int ncol, uint8_t *__restrict__ out,
    int64_t out_stride, bool wide) {
    constexpr int ROWS = TM + TN, WM = TM / 2, WN = TN / 2, MI = WM / 16, NI = WN / 16;
    constexpr int LOADS = ROWS * 8 / kTileThreads;        // 16-byte pieces of a stage a thread loads
    constexpr int SLOADS = ROWS * 2 / kTileThreads;       // scale words (four blocks) of a stage
    __shared__ __align__(1024) uint8_t codes[2][ROWS * 128];
    __shared__ __align__(16) uint32_t scales[2][ROWS * 2];

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
    const uint8_t *wsc = w_scales + (int64_t)g * O * nblk;
    const uint8_t *asc = a_scales + first * nblk;
    const __amdgpu_buffer_rsrc_t a_src = rsrc(a_codes + first * pitch, (int64_t)rows * pitch);
    const __amdgpu_buffer_rsrc_t w_src = rsrc(w_codes + (int64_t)g * O * pitch, (int64_t)O * pitch);

    // Row of the weights behind tile row j: plain, neighbours; gated, each wave's half of the tile has its gate
    // rows first, then the up rows of the same outputs. Rows past the end repeat the last one.
    const auto weight_row = [&](int j) {
        if (!GATED) return min(o0 + j, width - 1);
        const int half = j / WN, jj = j % WN;
        const int o = min(o0 + half * (WN / 2) + jj % (WN / 2), width - 1);
        return jj < WN / 2 ? o : width + o;
    };

    // Piece l of a stage: tile row (l * 256 + tid) / 8, held at place tid % 8 of its 128 bytes; place p of row r
    // holds block p ^ (r & 7), so that 16 rows' reads of one block spread over the banks.
    const int place = tid & 7, r8 = tid >> 3, blk = place ^ (r8 & 7);
    int voff[LOADS];
#pragma unroll
    for (int l = 0; l < LOADS; ++l) {
        const int r = l * (kTileThreads / 8) + r8;
        voff[l] = (r < TM ? min(r, rows - 1) : weight_row(r - TM)) * pitch + blk * 16;
    }
    int soff[SLOADS];
#pragma unroll
    for (int l = 0; l < SLOADS; ++l) {
        const int r = (l * kTileThreads + tid) >> 1;
        soff[l] = (r < TM ? min(r, rows - 1) : weight_row(r - TM)) * nblk;
    }
    const int sword = tid & 1;

    const int stages = (nblk + kStageBlocks - 1) / kStageBlocks;
    const auto load_codes = [&](int st, int buf) {
        const bool past = st * kStageBlocks + blk >= nblk;  // blocks behind the row's end read as zero
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
            uint8_t *dst = &codes[buf][(l * kTileThreads + wave * 64) * 16];
            load_to_lds(l * (kTileThreads / 8) < TM ? a_src : w_src, dst, past ? 0x7FFFFFF0 : voff[l], st * 128);
        }
    };
    uint32_t sreg[SLOADS];
    const auto load_scales = [&](int st) {
        // the word of blocks b .. b + 3; at the row's end, the row's last four bytes (nblk >= 4) moved down, so
        // that blocks behind the end have scale byte 0
        const int b = st * kStageBlocks + 4 * sword, from = min(b, nblk - 4);
        const int down = min(8 * (b - from), 63);
#pragma unroll
        for (int l = 0; l < SLOADS; ++l) {
            const uint8_t *src = (((l * kTileThreads + tid) >> 1) < TM ? asc : wsc) + soff[l] + from;
            uint32_t v;
            __builtin_memcpy(&v, src, 4);
            sreg[l] = (uint32_t)((uint64_t)v >> down);
        }
    };
    const auto put_scales = [&](int buf) {
#pragma unroll
        for (int l = 0; l < SLOADS; ++l) scales[buf][l * kTileThreads + tid] = sreg[l];
    };

    f32x4 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    const int wm = (wave & 1) * WM, wn = TM + (wave >> 1) * WN;
    const int fr = lane & 15, q = lane >> 4;

    load_codes(0, 0);
    load_scales(0);
    put_scales(0);
    __syncthreads();
    for (int st = 0; st < stages; ++st) {
        const int buf = st & 1;
        i32x4 a[2][MI], w[2][NI];
        u32x2 as[MI], ws[NI];
#pragma unroll
        for (int i = 0; i < MI; ++i) as[i] = *reinterpret_cast<const u32x2 *>(&scales[buf][(wm + i * 16 + fr) * 2]);
#pragma unroll
        for (int j = 0; j < NI; ++j) ws[j] = *reinterpret_cast<const u32x2 *>(&scales[buf][(wn + j * 16 + fr) * 2]);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const int at = ((4 * ks + q) ^ (fr & 7)) * 16;
#pragma unroll
            for (int i = 0; i < MI; ++i)
                a[ks][i] = *reinterpret_cast<const i32x4 *>(&codes[buf][(wm + i * 16 + fr) * 128 + at]);
#pragma unroll
            for (int j = 0; j < NI; ++j)
                w[ks][j] = *reinterpret_cast<const i32x4 *>(&codes[buf][(wn + j * 16 + fr) * 128 + at]);
        }
        if (st + 1 < stages) {
            load_codes(st + 1, buf ^ 1);
            load_scales(st + 1);
        }
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const int sa = (int)(as[i][ks] >> (8 * q));
#pragma unroll
                for (int j = 0; j < NI; ++j)
                    acc[i][j] = mfma(w[ks][j], (int)(ws[j][ks] >> (8 * q)), a[ks][i], sa, acc[i][j]);
            }
        }
        // the wait for the next stage stays behind this stage's products
        __builtin_amdgcn_sched_barrier(0);
        if (st + 1 < stages) put_scales(buf ^ 1);
        __syncthreads();
    }

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
            store4(dst, o0 + (wave >> 1) * (GATED ? WN / 2 : WN) + j * 16 + 4 * q, width, wide, v);
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

template <int TM, int TN>
hipError_t tiles(const void *a_codes, const void *a_scales, int64_t a_rows, const int32_t *group_base,
                 int32_t G, const void *w_codes, const void *w_scales, int32_t O, int32_t H, bool gated,
                 void *out, int64_t out_stride, bool wide, hipStream_t stream) {
    const int width = gated ? O / 2 : O, tn = gated ? TN / 2 : TN;
    const int ncol = (width + tn - 1) / tn;
    const int64_t row_tiles = a_rows / TM + (a_rows < G ? a_rows : G);  // at most
    const int64_t grid = (row_tiles * ncol + 7) / 8 * 8;
    auto *kernel = gated ? product_tile_kernel<TM, TN, true> : product_tile_kernel<TM, TN, false>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(kTileThreads), 0, stream,
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
    if (mean >= 192 && H >= 128)
        return tiles<256, 256>(a_codes, a_scales, a_rows, group_base, G, w_codes, w_scales, O, H, gated, out,
                               out_stride_bytes, wide, stream);
    if (mean >= 32 && H >= 128)
        return tiles<128, 128>(a_codes, a_scales, a_rows, group_base, G, w_codes, w_scales, O, H, gated, out,
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
