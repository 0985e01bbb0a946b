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

}  // namespace

hipError_t launch_mx_product(const void *a_codes, const void *a_scales, int64_t a_rows,
                             const int32_t *group_base, int32_t G, const void *w_codes,
                             const void *w_scales, int32_t O, int32_t H, int32_t epilogue, void *out,
                             int64_t out_stride_bytes, hipStream_t stream) {
    if (a_rows == 0) return hipSuccess;
    const bool gated = epilogue == MOE_MX_GATED;
    const int width = gated ? O / 2 : O;
    const int64_t tiles = a_rows / 16 + (a_rows < G ? a_rows : G);
    auto *kernel = gated ? product_kernel<true> : product_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)tiles, (width + 15) / 16), dim3(64), 0, stream,
                       static_cast<const uint8_t *>(a_codes), static_cast<const uint8_t *>(a_scales),
                       a_rows, group_base, G, static_cast<const uint8_t *>(w_codes),
                       static_cast<const uint8_t *>(w_scales), O, H, static_cast<uint8_t *>(out),
                       out_stride_bytes);
    return hipGetLastError();
}

}  // namespace moe
