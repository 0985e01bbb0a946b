// MX rows for gfx950: bf16 rows to microscaled blocks (E2M1 or E4M3 codes, one scale byte for 32 values) and
// back (mx_blocks.h has the arithmetic).
//
// Both directions are streams: 2 bytes a value on the bf16 side, 17/32 or 33/32 on the other. A lane takes
// eight values (16 bytes of bf16), four lanes a block, whose largest magnitude two DPP steps give to all
// four; a one-wave workgroup takes two such vectors a lane of one row, loads first. Measured at 32768 rows of
// 7168, E2M1 there and back, E4M3 there and back (us): 91.9, 96.7, 108, 111 (6.1 to 6.6 TB/s); one vector a
// lane 101, 119, 108, 111; four 98, 106, 116, 118; 128 lanes 95.6, 99.2, 114, 117; with the caches' default
// policies 101, 101, 118, 117.

#include "mx_blocks.h"

namespace moe {
namespace {

using namespace mx;

constexpr int kPartThreads = 64;
constexpr int kVecs = 2;                   // vectors of a lane
constexpr int kLoadPolicy = 2;             // nt
constexpr int kStorePolicy = 1 | 16 | 2;   // sc0 sc1 nt

__device__ inline __amdgpu_buffer_rsrc_t rsrc(const void *base, int32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, bytes, 0x00020000);
}

__device__ inline int64_t row_count(const int32_t *num_rows, int64_t max_rows) {
    if (!num_rows) return max_rows;
    const int64_t n = *num_rows;
    return n < 0 ? 0 : min(n, max_rows);
}

// grid = max_rows * nparts; workgroup (r, q) takes vectors [q, q + 1) * kVecs * kPartThreads of row r, nvec =
// H / 8, a multiple of 4, so that a block's four lanes are in the row or behind it together. The loads are issued
// before the count arrives: every row below max_rows lies in the buffer.
template <int FORMAT>
__global__ __launch_bounds__(kPartThreads) void mx_quantize_kernel(
    const uint8_t *__restrict__ rows, int64_t stride, const int32_t *__restrict__ num_rows,
    int64_t max_rows, int nvec, int nparts, uint8_t *__restrict__ codes,
    uint8_t *__restrict__ scales) {
    constexpr int kCode = FORMAT == MOE_MX_E2M1 ? 4 : 8;  // code bytes of eight values
    const int64_t r = blockIdx.x / nparts;
    const int v0 = (int)(blockIdx.x - r * nparts) * kVecs * kPartThreads + threadIdx.x;
    const __amdgpu_buffer_rsrc_t src = rsrc(rows + r * stride, nvec << 4);
    u32x4 x[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
        x[i] = __builtin_amdgcn_raw_buffer_load_b128(src, (v0 + i * kPartThreads) << 4, 0, kLoadPolicy);
    if (r >= row_count(num_rows, max_rows)) return;
    const __amdgpu_buffer_rsrc_t dst = rsrc(codes + r * nvec * kCode, nvec * kCode);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int v = v0 + i * kPartThreads;
        const uint32_t byte = scale_byte<FORMAT>(max_of_four_lanes(amax_bits(x[i])));
        const u32x2 c = encode<FORMAT>(x[i], byte);
        if constexpr (FORMAT == MOE_MX_E2M1)
            __builtin_amdgcn_raw_buffer_store_b32(c.x, dst, v << 2, 0, kStorePolicy);
        else
            __builtin_amdgcn_raw_buffer_store_b64(c, dst, v << 3, 0, kStorePolicy);
        if ((threadIdx.x & 3) == 0 && v < nvec) scales[(r * nvec + v) >> 2] = (uint8_t)byte;
    }
}

// The way back, same grid.
template <int FORMAT>
__global__ __launch_bounds__(kPartThreads) void mx_dequantize_kernel(
    const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
    const int32_t *__restrict__ num_rows, int64_t max_rows, int nvec, int nparts,
    uint8_t *__restrict__ rows, int64_t stride) {
    constexpr int kCode = FORMAT == MOE_MX_E2M1 ? 4 : 8;
    const int64_t r = blockIdx.x / nparts;
    const int v0 = (int)(blockIdx.x - r * nparts) * kVecs * kPartThreads + threadIdx.x;
    const __amdgpu_buffer_rsrc_t src = rsrc(codes + r * nvec * kCode, nvec * kCode);
    const __amdgpu_buffer_rsrc_t scale_src = rsrc(scales + r * (nvec >> 2), nvec >> 2);
    u32x2 c[kVecs];
    uint32_t byte[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int v = v0 + i * kPartThreads;
        if constexpr (FORMAT == MOE_MX_E2M1)
            c[i] = u32x2{__builtin_amdgcn_raw_buffer_load_b32(src, v << 2, 0, kLoadPolicy), 0u};
        else
            c[i] = __builtin_amdgcn_raw_buffer_load_b64(src, v << 3, 0, kLoadPolicy);
        byte[i] = __builtin_amdgcn_raw_buffer_load_b8(scale_src, v >> 2, 0, 0);
    }
    if (r >= row_count(num_rows, max_rows)) return;
    const __amdgpu_buffer_rsrc_t dst = rsrc(rows + r * stride, nvec << 4);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        float f[8];
        if constexpr (FORMAT == MOE_MX_E2M1) decode_e2m1(c[i].x, scale_value(byte[i]), f);
        else decode_e4m3(c[i], scale_value(byte[i]), f);
        u32x4 out;
#pragma unroll
        for (int w = 0; w < 4; ++w) out[w] = bf16_pair(f[2 * w], f[2 * w + 1]);
        __builtin_amdgcn_raw_buffer_store_b128(out, dst, (v0 + i * kPartThreads) << 4, 0, kStorePolicy);
    }
}

}  // namespace

hipError_t launch_mx_quantize(const void *rows, int64_t row_stride_bytes, const int32_t *num_rows,
                              int64_t max_rows, int32_t H, int32_t format, void *codes,
                              void *scales, hipStream_t stream) {
    if (max_rows == 0) return hipSuccess;
    const int nvec = H / 8;
    const int nparts = (nvec + kVecs * kPartThreads - 1) / (kVecs * kPartThreads);
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
    const int nparts = (nvec + kVecs * kPartThreads - 1) / (kVecs * kPartThreads);
    auto *kernel =
        format == MOE_MX_E2M1 ? mx_dequantize_kernel<MOE_MX_E2M1> : mx_dequantize_kernel<MOE_MX_E4M3>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(max_rows * nparts)), dim3(kPartThreads), 0, stream,
                       static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales),
                       num_rows, max_rows, nvec, nparts, static_cast<uint8_t *>(rows), row_stride_bytes);
    return hipGetLastError();
}

}  // namespace moe
