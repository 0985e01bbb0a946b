// Rows to 8 bits with one fp32 scale a row, and back, for gfx950 (see moe_row_quantize in moe.h; row_codes.h has the
// arithmetic, the quantised dispatch's).
//
// Both directions are streams that HBM bounds: 32768 rows of 7168 to INT8 and back, 705 MB each, take 118 and 115 us (6.0 and
// 6.1 TB/s; a large copy reaches 6.7). The quotients' corrections count on the way there. In loops of calls, 121 as it is, the
// same rows took 131 with a clamp, the zeros' signs and a conversion for each, 157 with an uncorrected product and a division
// where it comes near a border (bf16 rows often hold half of their largest value, halfway between two codes), and 143 as a
// row over 448 lanes of two neighbouring vectors, reduced by shuffles. On the way back one vector a lane takes 122.

#include "row_codes.h"
#include "wave_ops.h"

namespace moe {
namespace {

using mx::bf16_pair;
using mx::u32x2;
using rows::u32x4;

constexpr int kMaxThreads = 512;  // of a workgroup that takes a row
constexpr int kRowsAlone = 4;      // rows of a workgroup whose waves take one each
constexpr int kPartThreads = 64;
constexpr int kVecs = 2;                       // vectors of a lane on the way back
constexpr int kLoadPolicy = 2;                 // nt
constexpr int kStorePolicy = 2;                // nt
constexpr int kWideStorePolicy = 1 | 16 | 2;   // sc0 sc1 nt

__device__ inline int64_t row_count(const int32_t *num_rows, int64_t max_rows) {
    if (!num_rows) return max_rows;
    const int64_t n = *num_rows;
    return n < 0 ? 0 : min(n, max_rows);
}

// A workgroup a row, or a wave a row (waves == 1), vectors u + i * lanes of 8 values a lane. The largest magnitude is taken
// on bf16 bits, where infinities and NaNs are above all numbers. The loads are issued before the count arrives: every
// row below max_rows lies in the buffer.
template <int VPL, int QUANT>
__global__ __launch_bounds__(kMaxThreads) void row_quantize_kernel(
    const uint8_t *__restrict__ rows, int64_t stride, const int32_t *__restrict__ num_rows, int64_t max_rows,
    int nvec, int waves, uint8_t *__restrict__ codes, float *__restrict__ scales) {
    __shared__ uint32_t wave_top[kMaxThreads / 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool alone = waves == 1;
    const int lanes = waves << 6, u = alone ? lane : (int)threadIdx.x;
    const int64_t r = alone ? (int64_t)blockIdx.x * kRowsAlone + wave : blockIdx.x;
    if (r >= max_rows) return;
    const __amdgpu_buffer_rsrc_t src = rows::rsrc(rows + r * stride, nvec << 4);
    u32x4 x[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] = __builtin_amdgcn_raw_buffer_load_b128(src, (u + i * lanes) << 4, 0, kLoadPolicy);
    if (r >= row_count(num_rows, max_rows)) return;
    uint32_t top = mx::amax_bits(x[0]);
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = max(top, mx::amax_bits(x[i]));
    top = wave::most(top);
    if (!alone) {
        if (lane == 0) wave_top[wave] = top;
        __syncthreads();
        for (int w = 0; w < waves; ++w) top = max(top, wave_top[w]);
    }
    const float scale = top >= 0x7F80u ? __uint_as_float(0x7FC00000u)
                                       : __uint_as_float(top << 16) / rows::code_max<QUANT>();
    const bool fast = rows::corrected(scale);
    const float inv = 1.0f / scale;
    const __amdgpu_buffer_rsrc_t dst = rows::rsrc(codes + r * (nvec << 3), nvec << 3);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        float v[8];
#pragma unroll
        for (int w = 0; w < 4; ++w) v[2 * w] = rows::bf16_lo(x[i][w]), v[2 * w + 1] = rows::bf16_hi(x[i][w]);
        u32x2 c = {0u, 0u};
        if (fast) c = rows::codes8<QUANT>(v, scale, inv);
        else if (scale > 0.0f) c = rows::divided8<QUANT>(v, scale);
        __builtin_amdgcn_raw_buffer_store_b64(c, dst, (u + i * lanes) << 3, 0, kStorePolicy);
    }
    if (u == 0) scales[r] = scale;
}

template <int QUANT>
__device__ inline void values4(uint32_t codes, float scale, float (&v)[4]) {
    if constexpr (QUANT == MOE_QUANT_FP8_E4M3_DYN) {
        const mx::f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false);
        const mx::f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
        v[0] = a.x * scale; v[1] = a.y * scale;
        v[2] = b.x * scale; v[3] = b.y * scale;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(codes >> (8 * i)) * scale;
    }
}

// grid = max_rows * nparts; workgroup (r, q) takes vectors [q, q + 1) * kVecs * kPartThreads of row r.
template <int QUANT>
__global__ __launch_bounds__(kPartThreads) void row_dequantize_kernel(
    const uint8_t *__restrict__ codes, const float *__restrict__ scales, const int32_t *__restrict__ num_rows,
    int64_t max_rows, int nvec, int nparts, uint8_t *__restrict__ rows, int64_t stride) {
    const int64_t r = blockIdx.x / nparts;
    const int v0 = (int)(blockIdx.x - r * nparts) * kVecs * kPartThreads + threadIdx.x;
    const __amdgpu_buffer_rsrc_t src = rows::rsrc(codes + r * (nvec << 3), nvec << 3);
    u32x2 c[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
        c[i] = __builtin_amdgcn_raw_buffer_load_b64(src, (v0 + i * kPartThreads) << 3, 0, kLoadPolicy);
    const float scale = scales[r];
    if (r >= row_count(num_rows, max_rows)) return;
    const __amdgpu_buffer_rsrc_t dst = rows::rsrc(rows + r * stride, nvec << 4);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        float lo[4], hi[4];
        values4<QUANT>(c[i].x, scale, lo);
        values4<QUANT>(c[i].y, scale, hi);
        const u32x4 out = {bf16_pair(lo[0], lo[1]), bf16_pair(lo[2], lo[3]), bf16_pair(hi[0], hi[1]), bf16_pair(hi[2], hi[3])};
        __builtin_amdgcn_raw_buffer_store_b128(out, dst, (v0 + i * kPartThreads) << 4, 0, kWideStorePolicy);
    }
}

}  // namespace

hipError_t launch_row_quantize(const void *rows, int64_t row_stride_bytes, const int32_t *num_rows,
                               int64_t max_rows, int32_t H, int32_t quant, void *codes,
                               float *scales, hipStream_t stream) {
    if (max_rows == 0) return hipSuccess;
    const int nvec = H / 8, waves = row_waves(H);
    const auto pick = [&](auto type) {
        constexpr int Q = decltype(type)::value;
        return nvec <= 64 ? row_quantize_kernel<1, Q> : nvec <= 1024 ? row_quantize_kernel<2, Q> : row_quantize_kernel<4, Q>;
    };
    auto *kernel = quant == MOE_QUANT_INT8_DYN ? pick(std::integral_constant<int, MOE_QUANT_INT8_DYN>{})
                                               : pick(std::integral_constant<int, MOE_QUANT_FP8_E4M3_DYN>{});
    const int64_t grid = waves == 1 ? (max_rows + kRowsAlone - 1) / kRowsAlone : max_rows;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(64 * (waves == 1 ? kRowsAlone : waves)), 0, stream,
                       static_cast<const uint8_t *>(rows), row_stride_bytes, num_rows, max_rows, nvec, waves,
                       static_cast<uint8_t *>(codes), scales);
    return hipGetLastError();
}

hipError_t launch_row_dequantize(const void *codes, const float *scales, const int32_t *num_rows,
                                 int64_t max_rows, int32_t H, int32_t quant, void *rows,
                                 int64_t row_stride_bytes, hipStream_t stream) {
    if (max_rows == 0) return hipSuccess;
    const int nvec = H / 8, nparts = (nvec + kVecs * kPartThreads - 1) / (kVecs * kPartThreads);
    auto *kernel = quant == MOE_QUANT_INT8_DYN ? row_dequantize_kernel<MOE_QUANT_INT8_DYN>
                                               : row_dequantize_kernel<MOE_QUANT_FP8_E4M3_DYN>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(max_rows * nparts)), dim3(kPartThreads), 0, stream,
                       static_cast<const uint8_t *>(codes), scales, num_rows, max_rows, nvec, nparts,
                       static_cast<uint8_t *>(rows), row_stride_bytes);
    return hipGetLastError();
}

}  // namespace moe
