// The experts' product of INT8 rows and weights for gfx950 (see moe_int8_product in moe.h).
//
// v_mfma_i32_16x16x64_i8 multiplies a 16 x 64 by a 64 x 16 tile, lane l giving 16 consecutive values (16 bytes) of row
// l % 16, k-block l / 16, of either operand. The weights are the first operand, so that a lane's four results are
// neighbouring outputs of one row. Sums are whole numbers below 2^31 (H * 128 * 128 <= 2^28), the same in any order.

#include "product_rows.h"

namespace moe {
namespace {

using namespace product;

typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ inline i32x4 mfma(const i32x4 &a, const i32x4 &b, const i32x4 &c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// A wave takes 16 rows of a group and 32 weight rows (16 outputs when GATED).
template <bool GATED>
__global__ __launch_bounds__(64) void product_kernel(const uint8_t *__restrict__ a_codes, const float *__restrict__ a_scales, int64_t a_rows,
                                                     const int32_t *__restrict__ base, int G, const uint8_t *__restrict__ w_codes,
                                                     const float *__restrict__ w_scales, int O, int H, uint8_t *__restrict__ out, int64_t out_stride) {
    int g;
    int64_t first, last;
    if (!find_rows<16>(base, G, a_rows, blockIdx.x, g, first, last)) return;
    g = __builtin_amdgcn_readfirstlane(g);
    first = __builtin_amdgcn_readfirstlane((int)first);
    last = __builtin_amdgcn_readfirstlane((int)last);
    const int lane = threadIdx.x & 63, fr = lane & 15, q = lane >> 4, rows = (int)(last - first);
    const int width = GATED ? O / 2 : O, o0 = blockIdx.y * (GATED ? 16 : 32);
    const uint8_t *arow = a_codes + (first + min(fr, rows - 1)) * H;
    const uint8_t *wrow[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int o = GATED ? min(o0 + fr, width - 1) + j * width : min(o0 + 16 * j + fr, width - 1);
        wrow[j] = w_codes + ((int64_t)g * O + o) * H;
    }
    i32x4 acc[2] = {i32x4{0, 0, 0, 0}, i32x4{0, 0, 0, 0}};
    for (int k = 0; k < H; k += 64) {
        const int at = k + 16 * q;
        i32x4 a = {0, 0, 0, 0}, w[2] = {a, a};
        if (at < H) {
            a = *reinterpret_cast<const i32x4 *>(arow + at);
            w[0] = *reinterpret_cast<const i32x4 *>(wrow[0] + at);
            w[1] = *reinterpret_cast<const i32x4 *>(wrow[1] + at);
        }
        acc[0] = mfma(w[0], a, acc[0]);
        acc[1] = mfma(w[1], a, acc[1]);
    }
    if (fr >= rows) return;
    const float sa = a_scales[first + fr];
    const float *sw = w_scales + (int64_t)g * O;
    uint16_t *dst = reinterpret_cast<uint16_t *>(out + (first + fr) * out_stride);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (GATED) {
            const int o = o0 + 4 * q + e;
            if (o >= width) continue;
            const float gate = (float)acc[0][e] * sa * sw[o], up = (float)acc[1][e] * sa * sw[width + o];
            dst[o] = (uint16_t)bf16_pair(silu_times(gate, up), 0.0f);
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int o = o0 + 16 * j + 4 * q + e;
                if (o < width) dst[o] = (uint16_t)bf16_pair((float)acc[j][e] * sa * sw[o], 0.0f);
            }
        }
    }
}

}  // namespace

hipError_t launch_int8_product(const void *a_codes, const float *a_scales, int64_t a_rows,
                               const int32_t *group_base, int32_t G, const void *w_codes,
                               const float *w_scales, int32_t O, int32_t H, int32_t epilogue,
                               void *out, int64_t out_stride_bytes, hipStream_t stream) {
    if (a_rows == 0) return hipSuccess;
    const bool gated = epilogue == MOE_MX_GATED;
    const int64_t row_tiles = a_rows / 16 + (a_rows < G ? a_rows : G);  // at most
    const int ncol = gated ? (O / 2 + 15) / 16 : (O + 31) / 32;
    auto *kernel = gated ? product_kernel<true> : product_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)row_tiles, ncol), dim3(64), 0, stream, static_cast<const uint8_t *>(a_codes),
                       a_scales, a_rows, group_base, G, static_cast<const uint8_t *>(w_codes), w_scales, O, H,
                       static_cast<uint8_t *>(out), out_stride_bytes);
    return hipGetLastError();
}

}  // namespace moe
