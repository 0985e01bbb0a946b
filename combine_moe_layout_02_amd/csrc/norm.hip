// The residual's addition and the root-mean-square norm, with its output in bf16, in 8 bits or both, and its gradients, for
// gfx950 (see moe_rms_norm in moe.h).
//
// A workgroup takes a row: its lanes hold it in registers from the load to the store, vector v = lane + i * blockDim of 8
// values, so that every byte is moved once. The sum of squares is taken in 64 bits: the squares of bf16 values are exact
// there, nothing overflows, and the codes, which lie next to borders, do not depend on the order of the additions.

#include "mx_blocks.h"
#include "pack_rows.h"

namespace moe {
namespace {

using mx::bf16_hi;
using mx::bf16_lo;
using mx::bf16_pair;
using mx::u32x2;
using mx::u32x4;

constexpr int kMaxWaves = 16;

// 8 neighbouring weights; vectors past the row are not read.
template <int WTYPE>
__device__ inline void load_weights(__amdgpu_buffer_rsrc_t src, int v, float (&w)[8]) {
    if constexpr (WTYPE == MOE_BF16) {
        const u32x4 b = rows::load16(src, v << 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[2 * i] = bf16_lo(b[i]), w[2 * i + 1] = bf16_hi(b[i]);
    } else {
        const u32x4 a = rows::load16(src, v << 5), b = rows::load16(src, (v << 5) + 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __uint_as_float(a[i]), w[4 + i] = __uint_as_float(b[i]);
    }
}

template <int WTYPE>
__device__ inline __amdgpu_buffer_rsrc_t weight_rsrc(const void *weight, int nvec) {
    return rows::rsrc(weight, nvec << (WTYPE == MOE_BF16 ? 4 : 5));
}

__device__ inline double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// fp32(1 / sqrt(sum / H + eps))
__device__ inline float inverse_rms(double sum, int H, float eps) {
    return (float)(1.0 / sqrt(sum / (double)H + (double)eps));
}

// RN(1 / scale) and the corrections of div_by_scale give the correctly rounded quotient unless all bits of the scale's
// mantissa are set.
__device__ inline bool fast_scale(float scale) {
    return scale >= rows::kFastDivMinScale && scale <= 0x1.fffffep127f &&
           (__float_as_uint(scale) & 0x7FFFFFu) != 0x7FFFFFu;
}

template <int QUANT, bool FAST>
__device__ inline uint32_t code4(const float *v, float scale, float y) {
    const float q0 = rows::quotient<FAST>(v[0], scale, y), q1 = rows::quotient<FAST>(v[1], scale, y);
    const float q2 = rows::quotient<FAST>(v[2], scale, y), q3 = rows::quotient<FAST>(v[3], scale, y);
    if constexpr (QUANT == MOE_QUANT_FP8_E4M3_DYN)
        return rows::e4m3fn_pack4(q0, q1, q2, q3);
    else
        return rows::int8_code(q0) | (rows::int8_code(q1) << 8) | (rows::int8_code(q2) << 16) | (rows::int8_code(q3) << 24);
}

// grid = rows. sum may be x's or residual's rows: a lane stores what it has read.
template <int VPL, int QUANT, int WTYPE>
__global__ __launch_bounds__(1024) void rms_norm_kernel(const uint8_t *x, int64_t x_stride, const uint8_t *residual,
                                                        int64_t residual_stride, const uint8_t *__restrict__ weight, float eps,
                                                        int nvec, uint8_t *sum, int64_t sum_stride, uint8_t *__restrict__ out,
                                                        uint8_t *__restrict__ codes, float *__restrict__ scales) {
    __shared__ double part[kMaxWaves];
    __shared__ float wave_max[kMaxWaves];
    const int64_t r = blockIdx.x;
    const int u = threadIdx.x, lane = u & 63, wave = u >> 6, waves = blockDim.x >> 6, row_bytes = nvec << 4;
    const __amdgpu_buffer_rsrc_t src = rows::rsrc(x + r * x_stride, row_bytes);
    u32x4 h[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) h[i] = rows::load16(src, (u + i * blockDim.x) << 4);
    if (residual) {
        const __amdgpu_buffer_rsrc_t add = rows::rsrc(residual + r * residual_stride, row_bytes);
        const __amdgpu_buffer_rsrc_t dst = rows::rsrc(sum + r * sum_stride, row_bytes);
        u32x4 a[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) a[i] = rows::load16(add, (u + i * blockDim.x) << 4);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
#pragma unroll
            for (int w = 0; w < 4; ++w)
                h[i][w] = bf16_pair(bf16_lo(h[i][w]) + bf16_lo(a[i][w]), bf16_hi(h[i][w]) + bf16_hi(a[i][w]));
            __builtin_amdgcn_raw_buffer_store_b128(h[i], dst, (u + i * blockDim.x) << 4, 0, 0);
        }
    }
    double square = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const double lo = bf16_lo(h[i][w]), hi = bf16_hi(h[i][w]);
            square = fma(lo, lo, square);
            square = fma(hi, hi, square);
        }
    }
    square = wave_sum(square);
    if (lane == 0) part[wave] = square;
    __syncthreads();
    square = part[0];
    for (int w = 1; w < waves; ++w) square += part[w];
    const float rms = inverse_rms(square, nvec << 3, eps);

    const __amdgpu_buffer_rsrc_t wsrc = weight_rsrc<WTYPE>(weight, nvec);
    const __amdgpu_buffer_rsrc_t osrc = rows::rsrc(out + r * row_bytes, out ? row_bytes : 0);
    float y[VPL][8];
    float top = 0.0f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int v = u + i * blockDim.x;
        float wt[8];
        load_weights<WTYPE>(wsrc, v, wt);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float n = (e & 1 ? bf16_hi(h[i][e >> 1]) : bf16_lo(h[i][e >> 1])) * rms;
            y[i][e] = n * wt[e];
            if (v < nvec) {
                top = fmaxf(top, fabsf(y[i][e]));
                nan |= y[i][e] != y[i][e];
            }
        }
        if (out) {
            u32x4 o;
#pragma unroll
            for (int w = 0; w < 4; ++w) o[w] = bf16_pair(y[i][2 * w], y[i][2 * w + 1]);
            __builtin_amdgcn_raw_buffer_store_b128(o, osrc, v << 4, 0, 0);
        }
    }
    if constexpr (QUANT != MOE_QUANT_NONE) {
        if (nan) top = __uint_as_float(0x7F800000u);
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
        if (lane == 0) wave_max[wave] = top;
        __syncthreads();
        for (int w = 0; w < waves; ++w) top = fmaxf(top, wave_max[w]);
        const bool finite = top <= 0x1.fffffep127f;
        const float scale = finite ? top / rows::code_max<QUANT>() : __uint_as_float(0x7FC00000u);
        const bool fast = fast_scale(scale);
        const float inv = 1.0f / scale;
        const __amdgpu_buffer_rsrc_t dst = rows::rsrc(codes + r * (nvec << 3), nvec << 3);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            u32x2 c = {0u, 0u};
            if (fast)
                c = u32x2{code4<QUANT, true>(y[i], scale, inv), code4<QUANT, true>(y[i] + 4, scale, inv)};
            else if (scale > 0.0f)
                c = u32x2{code4<QUANT, false>(y[i], scale, inv), code4<QUANT, false>(y[i] + 4, scale, inv)};
            __builtin_amdgcn_raw_buffer_store_b64(c, dst, (u + i * blockDim.x) << 3, 0, 0);
        }
        if (u == 0) scales[r] = scale;
    }
}

// Part p of gridDim takes rows p, p + gridDim, ...; a lane's share of d_weight stays in registers until the end, where
// the part's sums go to partial[p].
template <int VPL, int WTYPE>
__global__ __launch_bounds__(1024) void rms_norm_backward_kernel(const uint8_t *__restrict__ dy, int64_t dy_stride, const uint8_t *__restrict__ sum, int64_t sum_stride,
                                                                 const uint8_t *__restrict__ weight, float eps, const uint8_t *__restrict__ d_sum, int64_t d_sum_stride,
                                                                 int64_t nrows, int nvec, uint8_t *__restrict__ dx, uint8_t *__restrict__ partial) {
    __shared__ double part[2][2][kMaxWaves];
    const int u = threadIdx.x, lane = u & 63, wave = u >> 6, waves = blockDim.x >> 6, row_bytes = nvec << 4;
    const __amdgpu_buffer_rsrc_t wsrc = weight_rsrc<WTYPE>(weight, nvec);
    float acc[VPL][8];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = 0.0f;
    int turn = 0;
    for (int64_t r = blockIdx.x; r < nrows; r += gridDim.x, turn ^= 1) {
        const __amdgpu_buffer_rsrc_t hsrc = rows::rsrc(sum + r * sum_stride, row_bytes);
        const __amdgpu_buffer_rsrc_t gsrc = rows::rsrc(dy + r * dy_stride, row_bytes);
        const __amdgpu_buffer_rsrc_t dsrc = rows::rsrc(d_sum + r * d_sum_stride, d_sum ? row_bytes : 0);
        u32x4 h[VPL], g[VPL], d[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int at = (u + i * blockDim.x) << 4;
            h[i] = rows::load16(hsrc, at);
            g[i] = rows::load16(gsrc, at);
            d[i] = rows::load16(dsrc, at);  // zero without d_sum
        }
        double square = 0.0, dot = 0.0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            float wt[8];
            load_weights<WTYPE>(wsrc, u + i * blockDim.x, wt);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double hv = e & 1 ? bf16_hi(h[i][e >> 1]) : bf16_lo(h[i][e >> 1]);
                const double gv = (double)(e & 1 ? bf16_hi(g[i][e >> 1]) : bf16_lo(g[i][e >> 1])) * (double)wt[e];
                square = fma(hv, hv, square);
                dot = fma(hv, gv, dot);
            }
        }
        square = wave_sum(square);
        dot = wave_sum(dot);
        if (lane == 0) part[turn][0][wave] = square, part[turn][1][wave] = dot;
        __syncthreads();
        square = part[turn][0][0], dot = part[turn][1][0];
        for (int w = 1; w < waves; ++w) square += part[turn][0][w], dot += part[turn][1][w];
        const int H = nvec << 3;
        const float rms = inverse_rms(square, H, eps);
        const float mean = (float)(dot * (double)rms / (double)H);  // of g * n
        const __amdgpu_buffer_rsrc_t dst = rows::rsrc(dx + r * row_bytes, row_bytes);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int v = u + i * blockDim.x;
            float wt[8], f[8];
            load_weights<WTYPE>(wsrc, v, wt);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n = (e & 1 ? bf16_hi(h[i][e >> 1]) : bf16_lo(h[i][e >> 1])) * rms;
                const float gy = e & 1 ? bf16_hi(g[i][e >> 1]) : bf16_lo(g[i][e >> 1]);
                acc[i][e] += gy * n;
                f[e] = rms * (gy * wt[e] - n * mean) + (e & 1 ? bf16_hi(d[i][e >> 1]) : bf16_lo(d[i][e >> 1]));
            }
            u32x4 o;
#pragma unroll
            for (int w = 0; w < 4; ++w) o[w] = bf16_pair(f[2 * w], f[2 * w + 1]);
            __builtin_amdgcn_raw_buffer_store_b128(o, dst, v << 4, 0, 0);
        }
    }
    const __amdgpu_buffer_rsrc_t psrc = rows::rsrc(partial + (int64_t)blockIdx.x * (nvec << 5), nvec << 5);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int at = (u + i * blockDim.x) << 5;
        const u32x4 lo = {__float_as_uint(acc[i][0]), __float_as_uint(acc[i][1]), __float_as_uint(acc[i][2]), __float_as_uint(acc[i][3])};
        const u32x4 hi = {__float_as_uint(acc[i][4]), __float_as_uint(acc[i][5]), __float_as_uint(acc[i][6]), __float_as_uint(acc[i][7])};
        __builtin_amdgcn_raw_buffer_store_b128(lo, psrc, at, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(hi, psrc, at + 16, 0, 0);
    }
}

// d_weight[h] = the parts' sums, in the order of 16 waves a sixteenth of them each: grid = H / 64 rounded up.
__global__ __launch_bounds__(1024) void norm_weight_kernel(const float *__restrict__ partial, int parts, int H,
                                                           float *__restrict__ d_weight) {
    __shared__ float sums[kMaxWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (h < H)
        for (int p = wave; p < parts; p += kMaxWaves) s += partial[(int64_t)p * H + h];
    sums[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || h >= H) return;
    for (int w = 1; w < kMaxWaves; ++w) s += sums[w][lane];
    d_weight[h] = s;
}

// Lanes of a row's workgroup: a vector each, as far as 1024 lanes go; H <= 16384 has 2048 vectors.
int row_threads(int nvec) { return nvec <= 1024 ? (nvec + 63) / 64 * 64 : ((nvec + 1) / 2 + 63) / 64 * 64; }

template <int QUANT, int WTYPE>
void norm(const uint8_t *x, int64_t x_stride, const uint8_t *residual, int64_t residual_stride, const uint8_t *weight, float eps, int64_t nrows,
          int nvec, uint8_t *sum, int64_t sum_stride, uint8_t *out, uint8_t *codes, float *scales, hipStream_t stream) {
    auto *kernel = nvec <= 1024 ? rms_norm_kernel<1, QUANT, WTYPE> : rms_norm_kernel<2, QUANT, WTYPE>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)nrows), dim3(row_threads(nvec)), 0, stream, x, x_stride, residual, residual_stride, weight, eps, nvec,
                       sum, sum_stride, out, codes, scales);
}

}  // namespace

hipError_t launch_rms_norm(const void *x, int64_t x_stride_bytes, const void *residual,
                           int64_t residual_stride_bytes, const void *weight, int32_t weight_type,
                           float eps, int64_t rows, int32_t H, int32_t quant, void *sum,
                           int64_t sum_stride_bytes, void *out, void *codes, float *scales,
                           hipStream_t stream) {
    if (rows == 0) return hipSuccess;
    const bool wide = weight_type == MOE_FP32;
    auto *call = quant == MOE_QUANT_NONE ? (wide ? norm<MOE_QUANT_NONE, MOE_FP32> : norm<MOE_QUANT_NONE, MOE_BF16>)
                 : quant == MOE_QUANT_INT8_DYN
                     ? (wide ? norm<MOE_QUANT_INT8_DYN, MOE_FP32> : norm<MOE_QUANT_INT8_DYN, MOE_BF16>)
                     : (wide ? norm<MOE_QUANT_FP8_E4M3_DYN, MOE_FP32> : norm<MOE_QUANT_FP8_E4M3_DYN, MOE_BF16>);
    call(static_cast<const uint8_t *>(x), x_stride_bytes, static_cast<const uint8_t *>(residual), residual_stride_bytes,
         static_cast<const uint8_t *>(weight), eps, rows, H / 8, static_cast<uint8_t *>(sum), sum_stride_bytes,
         static_cast<uint8_t *>(out), static_cast<uint8_t *>(codes), scales, stream);
    return hipGetLastError();
}

hipError_t launch_rms_norm_backward(const void *dy, int64_t dy_stride_bytes, const void *sum,
                                    int64_t sum_stride_bytes, const void *weight,
                                    int32_t weight_type, float eps, const void *d_sum,
                                    int64_t d_sum_stride_bytes, int64_t rows, int32_t H, void *dx,
                                    float *d_weight, void *workspace, hipStream_t stream) {
    const int nvec = H / 8, parts = (int)norm_parts(rows);
    if (rows > 0) {
        auto *kernel = weight_type == MOE_FP32
                           ? (nvec <= 1024 ? rms_norm_backward_kernel<1, MOE_FP32> : rms_norm_backward_kernel<2, MOE_FP32>)
                           : (nvec <= 1024 ? rms_norm_backward_kernel<1, MOE_BF16> : rms_norm_backward_kernel<2, MOE_BF16>);
        hipLaunchKernelGGL(kernel, dim3(parts), dim3(row_threads(nvec)), 0, stream, static_cast<const uint8_t *>(dy),
                           dy_stride_bytes, static_cast<const uint8_t *>(sum), sum_stride_bytes,
                           static_cast<const uint8_t *>(weight), eps, static_cast<const uint8_t *>(d_sum),
                           d_sum_stride_bytes, rows, nvec, static_cast<uint8_t *>(dx), static_cast<uint8_t *>(workspace));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(norm_weight_kernel, dim3((H + 63) / 64), dim3(1024), 0, stream,
                       static_cast<const float *>(workspace), parts, H, d_weight);
    return hipGetLastError();
}

}  // namespace moe
