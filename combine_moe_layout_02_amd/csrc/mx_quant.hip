// MX rows for gfx950: bf16 rows to microscaled blocks (E2M1 or E4M3 codes, one scale byte for 32 values) and
// back (mx_blocks.h has the arithmetic).
//
// Both directions are streams: 2 bytes a value on the bf16 side, 17/32 or 33/32 on the other. A lane takes
// eight values (16 bytes of bf16), four lanes a block, whose largest magnitude two DPP steps give to all
// four; a workgroup takes a part of one row.

#include "mx_blocks.h"

namespace moe {
namespace {

using namespace mx;

constexpr int kPartThreads = 64;

__device__ inline int64_t row_count(const int32_t *num_rows, int64_t max_rows) {
    if (!num_rows) return max_rows;
    const int64_t n = *num_rows;
    return n < 0 ? 0 : min(n, max_rows);
}

// grid = max_rows * nparts; workgroup (r, q) takes vectors [q, q + 1) * kPartThreads of row r, nvec = H / 8.
template <int FORMAT>
__global__ __launch_bounds__(kPartThreads) void mx_quantize_kernel(
    const uint8_t *__restrict__ rows, int64_t stride, const int32_t *__restrict__ num_rows,
    int64_t max_rows, int nvec, int nparts, uint8_t *__restrict__ codes,
    uint8_t *__restrict__ scales) {
    constexpr int kCode = FORMAT == MOE_MX_E2M1 ? 4 : 8;  // code bytes of eight values
    const int64_t r = blockIdx.x / nparts;
    const int q = (int)(blockIdx.x - r * nparts);
    if (r >= row_count(num_rows, max_rows)) return;
    const int v = q * kPartThreads + threadIdx.x;
    if (v >= nvec) return;  // nvec is a multiple of 4: a block's lanes leave or stay together
    const u32x4 x = *reinterpret_cast<const u32x4 *>(rows + r * stride + ((int64_t)v << 4));
    const uint32_t byte = scale_byte<FORMAT>(max_of_four_lanes(amax_bits(x)));
    const u32x2 c = encode<FORMAT>(x, byte);
    uint8_t *dst = codes + (r * nvec + v) * kCode;
    if constexpr (FORMAT == MOE_MX_E2M1) *reinterpret_cast<uint32_t *>(dst) = c.x;
    else *reinterpret_cast<u32x2 *>(dst) = c;
    if ((threadIdx.x & 3) == 0) scales[(r * nvec + v) >> 2] = (uint8_t)byte;
}

// The way back, same grid.
template <int FORMAT>
__global__ __launch_bounds__(kPartThreads) void mx_dequantize_kernel(
    const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
    const int32_t *__restrict__ num_rows, int64_t max_rows, int nvec, int nparts,
    uint8_t *__restrict__ rows, int64_t stride) {
    constexpr int kCode = FORMAT == MOE_MX_E2M1 ? 4 : 8;
    const int64_t r = blockIdx.x / nparts;
    const int q = (int)(blockIdx.x - r * nparts);
    if (r >= row_count(num_rows, max_rows)) return;
    const int v = q * kPartThreads + threadIdx.x;
    if (v >= nvec) return;
    const uint8_t *src = codes + (r * nvec + v) * kCode;
    const float scale = scale_value(scales[(r * nvec + v) >> 2]);
    float f[8];
    if constexpr (FORMAT == MOE_MX_E2M1) decode_e2m1(*reinterpret_cast<const uint32_t *>(src), scale, f);
    else decode_e4m3(*reinterpret_cast<const u32x2 *>(src), scale, f);
    u32x4 out;
#pragma unroll
    for (int w = 0; w < 4; ++w) out[w] = bf16_pair(f[2 * w], f[2 * w + 1]);
    *reinterpret_cast<u32x4 *>(rows + r * stride + ((int64_t)v << 4)) = out;
}

}  // namespace

hipError_t launch_mx_quantize(const void *rows, int64_t row_stride_bytes, const int32_t *num_rows,
                              int64_t max_rows, int32_t H, int32_t format, void *codes,
                              void *scales, hipStream_t stream) {
    if (max_rows == 0) return hipSuccess;
    const int nvec = H / 8;
    const int nparts = (nvec + kPartThreads - 1) / kPartThreads;
    auto *kernel = format == MOE_MX_E2M1 ? mx_quantize_kernel<MOE_MX_E2M1> : mx_quantize_kernel<MOE_MX_E4M3>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(max_rows * nparts)), dim3(kPartThreads), 0, stream,
                       static_cast<const uint8_t *>(rows), row_stride_bytes, num_rows, max_rows, nvec,
                       nparts, static_cast<uint8_t *>(codes), static_cast<uint8_t *>(scales));
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const void *codes, const void *scales, const int32_t *num_rows,
                                int64_t max_rows, int32_t H, int32_t format, void *rows,
                                int64_t row_stride_bytes, hipStream_t stream) {
    if (max_rows == 0) return hipSuccess;
    const int nvec = H / 8;
    const int nparts = (nvec + kPartThreads - 1) / kPartThreads;
    auto *kernel =
        format == MOE_MX_E2M1 ? mx_dequantize_kernel<MOE_MX_E2M1> : mx_dequantize_kernel<MOE_MX_E4M3>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(max_rows * nparts)), dim3(kPartThreads), 0, stream,
                       static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales),
                       num_rows, max_rows, nvec, nparts, static_cast<uint8_t *>(rows), row_stride_bytes);
    return hipGetLastError();
}

}  // namespace moe
