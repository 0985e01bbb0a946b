// Rows to 8 bits with one fp32 scale a row, and back, for gfx950 (see moe_row_quantize in moe.h; pack_rows.h has the
// arithmetic, which is the quantised dispatch's).

#include "mx_blocks.h"
#include "pack_rows.h"

namespace moe {
namespace {

using mx::bf16_pair;
using mx::u32x2;
using rows::u32x4;

__device__ inline int64_t row_count(const int32_t *num_rows, int64_t max_rows) {
    if (!num_rows) return max_rows;
    const int64_t n = *num_rows;
    return n < 0 ? 0 : min(n, max_rows);
}

// grid = max_rows; workgroup r takes row r, a lane 16 values (ngroups = H / 16 <= 1024). The largest magnitude is taken
// on bf16 bits, where infinities and NaNs are above all numbers.
template <int QUANT>
__global__ __launch_bounds__(1024) void row_quantize_kernel(
    const uint8_t *__restrict__ rows, int64_t stride, const int32_t *__restrict__ num_rows, int64_t max_rows,
    int ngroups, uint8_t *__restrict__ codes, float *__restrict__ scales) {
    __shared__ uint32_t wave_max[16];
    const int64_t r = blockIdx.x;
    const int u = threadIdx.x;
    const __amdgpu_buffer_rsrc_t src = rows::rsrc(rows + r * stride, ngroups << 5);
    const u32x4 a = rows::load16(src, u << 5), b = rows::load16(src, (u << 5) + 16);
    if (r >= row_count(num_rows, max_rows)) return;
    uint32_t top = max(mx::amax_bits(a), mx::amax_bits(b));
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d, 64));
    if ((u & 63) == 0) wave_max[u >> 6] = top;
    __syncthreads();
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) top = max(top, wave_max[w]);
    const float scale = top >= 0x7F80u ? __uint_as_float(0x7FC00000u)
                                       : __uint_as_float(top << 16) / rows::code_max<QUANT>();
    u32x4 c = {0u, 0u, 0u, 0u};
    if (top > 0 && top < 0x7F80u)
        c = scale >= rows::kFastDivMinScale ? rows::quant16<QUANT, true>(a, b, scale, 1.0f / scale)
                                            : rows::quant16<QUANT, false>(a, b, scale, 0.0f);
    const __amdgpu_buffer_rsrc_t dst = rows::rsrc(codes + r * (ngroups << 4), ngroups << 4);
    __builtin_amdgcn_raw_buffer_store_b128(c, dst, u << 4, 0, 0);
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

constexpr int kPartThreads = 64;

// grid = max_rows * nparts; workgroup (r, q) takes the q-th 64 groups of 8 values of row r.
template <int QUANT>
__global__ __launch_bounds__(kPartThreads) void row_dequantize_kernel(
    const uint8_t *__restrict__ codes, const float *__restrict__ scales, const int32_t *__restrict__ num_rows,
    int64_t max_rows, int nvec, int nparts, uint8_t *__restrict__ rows, int64_t stride) {
    const int64_t r = blockIdx.x / nparts;
    const int v = (int)(blockIdx.x - r * nparts) * kPartThreads + threadIdx.x;
    const __amdgpu_buffer_rsrc_t src = rows::rsrc(codes + r * (nvec << 3), nvec << 3);
    const u32x2 c = __builtin_amdgcn_raw_buffer_load_b64(src, v << 3, 0, 0);
    const float scale = scales[r];
    if (r >= row_count(num_rows, max_rows)) return;
    float lo[4], hi[4];
    values4<QUANT>(c.x, scale, lo);
    values4<QUANT>(c.y, scale, hi);
    const u32x4 out = {bf16_pair(lo[0], lo[1]), bf16_pair(lo[2], lo[3]), bf16_pair(hi[0], hi[1]), bf16_pair(hi[2], hi[3])};
    __builtin_amdgcn_raw_buffer_store_b128(out, rows::rsrc(rows + r * stride, nvec << 4), v << 4, 0, 0);
}

}  // namespace

hipError_t launch_row_quantize(const void *rows, int64_t row_stride_bytes, const int32_t *num_rows,
                               int64_t max_rows, int32_t H, int32_t quant, void *codes,
                               float *scales, hipStream_t stream) {
    if (max_rows == 0) return hipSuccess;
    auto *kernel = quant == MOE_QUANT_INT8_DYN ? row_quantize_kernel<MOE_QUANT_INT8_DYN>
                                               : row_quantize_kernel<MOE_QUANT_FP8_E4M3_DYN>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)max_rows), dim3((H / 16 + 63) / 64 * 64), 0, stream,
                       static_cast<const uint8_t *>(rows), row_stride_bytes, num_rows, max_rows, H / 16,
                       static_cast<uint8_t *>(codes), scales);
    return hipGetLastError();
}

hipError_t launch_row_dequantize(const void *codes, const float *scales, const int32_t *num_rows,
                                 int64_t max_rows, int32_t H, int32_t quant, void *rows,
                                 int64_t row_stride_bytes, hipStream_t stream) {
    if (max_rows == 0) return hipSuccess;
    const int nvec = H / 8, nparts = (nvec + kPartThreads - 1) / kPartThreads;
    auto *kernel = quant == MOE_QUANT_INT8_DYN ? row_dequantize_kernel<MOE_QUANT_INT8_DYN>
                                               : row_dequantize_kernel<MOE_QUANT_FP8_E4M3_DYN>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(max_rows * nparts)), dim3(kPartThreads), 0, stream,
                       static_cast<const uint8_t *>(codes), scales, num_rows, max_rows, nvec, nparts,
                       static_cast<uint8_t *>(rows), row_stride_bytes);
    return hipGetLastError();
}

}  // namespace moe
