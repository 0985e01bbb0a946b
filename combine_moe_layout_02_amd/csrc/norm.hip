// The residual's addition and the root-mean-square norm, with its output in bf16, in 8 bits or both, and its gradients, for
// gfx950 (see moe_rms_norm in moe.h).
//
// A workgroup takes a row, or a wave a short one: its lanes hold it in registers from the load to the store, vector v = lane +
// i * lanes of 8 values, so that every byte is moved once. The sum of squares is taken in 64 bits: the squares of bf16 values are
// exact there, nothing overflows, and the codes, which lie next to borders, do not depend on the order of the additions.
//
// HBM bounds the forward, and a row's chain the gradient. Call after call, 4096 rows of 7168, us and TB/s of what is read and
// written: to bf16 41.8 and 5.6, to INT8 38.5 and 5.3, the gradients 50.6 and 4.6 with d_weight's second kernel (4.7 of them). Two
// vectors a lane: to INT8 such rows take 38.5, with four 37.4, with eight 39.0, with one 55.6; 1531 rows of 2064 7.6, 8.5, 8.9 and
// 9.9; 4096 rows of 1024 7.5, 8.8, 12.1 and 9.2; 128 rows of 7168 5.1, 5.2, 5.8 and 6.2. Stores with nt (bf16, INT8) 41.8 and 38.5,
// with sc0 sc1 nt 42.0 and 38.8, written back 43.6 and 39.9. A workgroup that takes row after row with the weights in its
// registers and the next row's loads under way was no faster (44.9 where this form then took 42.0, two rows a compute unit in
// flight) and its registers cost short rows (1531 rows 9.9 to 14). Reductions through shuffles, an LDS access a step, and four
// times the waves a row took 72.

#include "row_codes.h"
#include "wave_ops.h"

namespace moe {
namespace {

using mx::bf16_hi;
using mx::bf16_lo;
using mx::bf16_pair;
using mx::u32x2;
using mx::u32x4;

constexpr int kLoadPolicy = 2;   // nt: rows are read once
constexpr int kStorePolicy = 2;  // nt

constexpr int kMaxWaves = 16;
constexpr int kMaxThreads = 512;  // of a workgroup that takes a row
constexpr int kRowsAlone = 4;      // rows of a workgroup whose waves take one each

__device__ inline u32x4 load16(__amdgpu_buffer_rsrc_t src, int off) {
    return __builtin_amdgcn_raw_buffer_load_b128(src, off, 0, kLoadPolicy);
}

// 8 neighbouring weights as they lie in memory; vectors past the row are zero.
template <int WTYPE>
struct Weights {
    u32x4 a, b;
    __device__ void load(__amdgpu_buffer_rsrc_t src, int v) {
        if constexpr (WTYPE == MOE_BF16) {
            a = rows::load16(src, v << 4);
        } else {
            a = rows::load16(src, v << 5);
            b = rows::load16(src, (v << 5) + 16);
        }
    }
    __device__ float value(int e) const {
        if constexpr (WTYPE == MOE_BF16) return e & 1 ? bf16_hi(a[e >> 1]) : bf16_lo(a[e >> 1]);
        else return __uint_as_float(e < 4 ? a[e & 3] : b[e & 3]);
    }
};

template <int WTYPE>
__device__ inline __amdgpu_buffer_rsrc_t weight_rsrc(const void *weight, int nvec) {
    return rows::rsrc(weight, nvec << (WTYPE == MOE_BF16 ? 4 : 5));
}

__device__ inline float value(const u32x4 &v, int e) { return e & 1 ? bf16_hi(v[e >> 1]) : bf16_lo(v[e >> 1]); }

// fp32(1 / sqrt(sum / H + eps))
__device__ inline float inverse_rms(double sum, int H, float eps) {
    return (float)(1.0 / sqrt(sum / (double)H + (double)eps));
}

// LDS accesses done, then all waves: loads and stores of memory stay in flight.
__device__ inline void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A workgroup a row, or a wave a row (waves == 1). sum may be x's or residual's rows: a lane stores what it has read.
template <int VPL, int QUANT, int WTYPE>
__global__ __launch_bounds__(kMaxThreads) void rms_norm_kernel(
    const uint8_t *x, int64_t x_stride, const uint8_t *residual, int64_t residual_stride,
    const uint8_t *__restrict__ weight, float eps, int64_t nrows, int nvec, int waves, uint8_t *sum,
    int64_t sum_stride, uint8_t *__restrict__ out, uint8_t *__restrict__ codes, float *__restrict__ scales) {
    __shared__ double part[kMaxWaves];
    __shared__ uint32_t wave_top[kMaxWaves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool alone = waves == 1;
    const int lanes = waves << 6, u = alone ? lane : (int)threadIdx.x, row_bytes = nvec << 4;
    const int64_t r = alone ? (int64_t)blockIdx.x * kRowsAlone + wave : blockIdx.x;
    if (r >= nrows) return;
    const __amdgpu_buffer_rsrc_t src = rows::rsrc(x + r * x_stride, row_bytes);
    u32x4 h[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) h[i] = load16(src, (u + i * lanes) << 4);
    u32x4 a[VPL];
    if (residual) {
        const __amdgpu_buffer_rsrc_t add = rows::rsrc(residual + r * residual_stride, row_bytes);
#pragma unroll
        for (int i = 0; i < VPL; ++i) a[i] = load16(add, (u + i * lanes) << 4);
    }
    Weights<WTYPE> wt[VPL];  // under way with the row, behind it
    const __amdgpu_buffer_rsrc_t wsrc = weight_rsrc<WTYPE>(weight, nvec);
#pragma unroll
    for (int i = 0; i < VPL; ++i) wt[i].load(wsrc, u + i * lanes);
    if (residual) {
        const __amdgpu_buffer_rsrc_t dst = rows::rsrc(sum + r * sum_stride, row_bytes);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
#pragma unroll
            for (int w = 0; w < 4; ++w)
                h[i][w] = bf16_pair(bf16_lo(h[i][w]) + bf16_lo(a[i][w]), bf16_hi(h[i][w]) + bf16_hi(a[i][w]));
            __builtin_amdgcn_raw_buffer_store_b128(h[i], dst, (u + i * lanes) << 4, 0, kStorePolicy);
        }
    }
    double square = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) square = fma((double)value(h[i], e), (double)value(h[i], e), square);
    square = wave::sum(square);
    if (!alone) {
        if (lane == 0) part[wave] = square;
        lds_barrier();
        square = part[0];
        for (int w = 1; w < waves; ++w) square += part[w];
    }
    const float rms = inverse_rms(square, nvec << 3, eps);

    float y[VPL][8];
    uint32_t top = 0;  // the largest magnitude's bits, where infinities and NaNs are above all numbers
#pragma unroll
    for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[i][e] = value(h[i], e) * rms * wt[i].value(e);
            if (QUANT != MOE_QUANT_NONE) top = max(top, __float_as_uint(y[i][e]) & 0x7FFFFFFFu);
        }
    if (out) {
        const __amdgpu_buffer_rsrc_t dst = rows::rsrc(out + r * row_bytes, row_bytes);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            u32x4 o;
#pragma unroll
            for (int w = 0; w < 4; ++w) o[w] = bf16_pair(y[i][2 * w], y[i][2 * w + 1]);
            __builtin_amdgcn_raw_buffer_store_b128(o, dst, (u + i * lanes) << 4, 0, kStorePolicy);
        }
    }
    if constexpr (QUANT != MOE_QUANT_NONE) {
        // a lane past the row has 0 * rms * 0, NaN where rms is one: then so are all the row's
        top = wave::most(top);
        if (!alone) {
            if (lane == 0) wave_top[wave] = top;
            lds_barrier();
            for (int w = 0; w < waves; ++w) top = max(top, wave_top[w]);
        }
        const float scale = top < 0x7F800000u ? __uint_as_float(top) / rows::code_max<QUANT>() : __uint_as_float(0x7FC00000u);
        const bool fast = rows::corrected(scale);
        const float inv = 1.0f / scale;
        const __amdgpu_buffer_rsrc_t dst = rows::rsrc(codes + r * (nvec << 3), nvec << 3);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            u32x2 c = {0u, 0u};
            if (fast) c = rows::codes8<QUANT>(y[i], scale, inv);
            else if (scale > 0.0f) c = rows::divided8<QUANT>(y[i], scale);
            __builtin_amdgcn_raw_buffer_store_b64(c, dst, (u + i * lanes) << 3, 0, kStorePolicy);
        }
        if (u == 0) scales[r] = scale;
    }
}

// Rows first, first + step, ..., a workgroup or a wave each, the next one's loads under way while one is turned; a lane's share of
// d_weight stays in registers until the end, where each workgroup's, or its waves', go to partial[part]. What bounds it is a
// row's chain with little beside it: two reductions in 64 bits, a barrier, then the divisions and the root, before the first
// store. Two vectors a lane need 162 registers (130 with fp32 weights), three waves a SIMD, so that of rows of 7168, seven waves
// each, one is on a compute unit at a time, and more parts than units are rounds and not rows at once: with bf16 weights 256
// parts 50.6 us for 4096 rows with the second kernel, 512 parts 53.8, 1024 57.0 (their sums are written and read again); 2048
// rows of 16384 55.4, 63.0 and 78.5. Shorter rows leave room for more: 4096 of 2048 23.9, 21.0 and 20.9, 4096 of 1024 21.8, 15.1
// and 14.4, 1531 of 2064 13.9, 13.7 and 16.3. fp32 weights take 49.8, 56.4, 21.5, 14.8 and 14.4 in the kept forms, 50.8, 55.7,
// 21.0, 14.5 and 13.7 where their products with dy were rounded before the mean. More rows' loads under way gain nothing: two,
// three and four ahead 51.3, 50.0 and 50.0 where one took 50.5. Several rows a workgroup, their shares of d_weight joined through
// LDS, took 52.7, and 1531 rows 18.4.
template <int VPL, int WTYPE>
__global__ __launch_bounds__(kMaxThreads) void rms_norm_backward_kernel(
    const uint8_t *__restrict__ dy, int64_t dy_stride, const uint8_t *__restrict__ sum, int64_t sum_stride,
    const uint8_t *__restrict__ weight, float eps, const uint8_t *__restrict__ d_sum, int64_t d_sum_stride,
    int64_t nrows, int nvec, int waves, uint8_t *__restrict__ dx, uint8_t *__restrict__ partial) {
    __shared__ double part[2][2][kMaxWaves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool alone = waves == 1;
    const int lanes = waves << 6, u = alone ? lane : (int)threadIdx.x, row_bytes = nvec << 4, H = nvec << 3;
    const int64_t step = alone ? (int64_t)gridDim.x * kRowsAlone : gridDim.x;
    const int64_t first = alone ? (int64_t)blockIdx.x * kRowsAlone + wave : blockIdx.x;
    Weights<WTYPE> wt[VPL];
    float acc[VPL][8];
    const __amdgpu_buffer_rsrc_t wsrc = weight_rsrc<WTYPE>(weight, nvec);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        wt[i].load(wsrc, u + i * lanes);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = 0.0f;
    }
    u32x4 nh[VPL], ng[VPL], nd[VPL];
    const auto load = [&](int64_t row) {
        const int bytes = row < nrows ? row_bytes : 0;
        const __amdgpu_buffer_rsrc_t hs = rows::rsrc(sum + row * sum_stride, bytes), gs = rows::rsrc(dy + row * dy_stride, bytes);
        const __amdgpu_buffer_rsrc_t ds = rows::rsrc(d_sum + row * d_sum_stride, d_sum ? bytes : 0);  // zero without d_sum
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int at = (u + i * lanes) << 4;
            nh[i] = load16(hs, at);
            ng[i] = load16(gs, at);
            nd[i] = load16(ds, at);
        }
    };
    load(first);
    int turn = 0;
    for (int64_t r = first; r < nrows; r += step, turn ^= 1) {
        u32x4 h[VPL], g[VPL], d[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) h[i] = nh[i], g[i] = ng[i], d[i] = nd[i];
        load(r + step);
        double square = 0.0, dot = 0.0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double hv = value(h[i], e);
                square = fma(hv, hv, square);
                // exact, as the sum may cancel: bf16 by bf16 in 32 bits, by fp32 in 64
                const double gw = WTYPE == MOE_BF16 ? (double)(value(g[i], e) * wt[i].value(e)) : (double)value(g[i], e) * (double)wt[i].value(e);
                dot = fma(hv, gw, dot);
            }
        square = wave::sum(square);
        dot = wave::sum(dot);
        if (!alone) {
            if (lane == 0) part[turn][0][wave] = square, part[turn][1][wave] = dot;
            lds_barrier();
            square = part[turn][0][0], dot = part[turn][1][0];
            for (int w = 1; w < waves; ++w) square += part[turn][0][w], dot += part[turn][1][w];
        }
        const float rms = inverse_rms(square, H, eps);
        const float mean = (float)(dot * (double)rms / (double)H);  // of g * n
        const __amdgpu_buffer_rsrc_t dst = rows::rsrc(dx + r * row_bytes, row_bytes);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n = value(h[i], e) * rms, gy = value(g[i], e);
                acc[i][e] += gy * n;
                f[e] = rms * (gy * wt[i].value(e) - n * mean) + value(d[i], e);
            }
            u32x4 o;
#pragma unroll
            for (int w = 0; w < 4; ++w) o[w] = bf16_pair(f[2 * w], f[2 * w + 1]);
            __builtin_amdgcn_raw_buffer_store_b128(o, dst, (u + i * lanes) << 4, 0, kStorePolicy);
        }
    }
    if (first >= nrows) return;  // a part of no rows has no place in the workspace
    const __amdgpu_buffer_rsrc_t psrc = rows::rsrc(partial + first * (nvec << 5), nvec << 5);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int at = (u + i * lanes) << 5;
        const u32x4 lo = {__float_as_uint(acc[i][0]), __float_as_uint(acc[i][1]), __float_as_uint(acc[i][2]), __float_as_uint(acc[i][3])};
        const u32x4 hi = {__float_as_uint(acc[i][4]), __float_as_uint(acc[i][5]), __float_as_uint(acc[i][6]), __float_as_uint(acc[i][7])};
        __builtin_amdgcn_raw_buffer_store_b128(lo, psrc, at, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(hi, psrc, at + 16, 0, 0);
    }
}

// d_weight[h] = the parts' sums: grid = H / 64 rounded up. A workgroup takes 64 columns, 16 lanes 16 bytes of each part; its
// lanes take every 64th part, and the 64 sums are added in order.
__global__ __launch_bounds__(1024) void norm_weight_kernel(const uint8_t *__restrict__ partial, int parts, int H,
                                                           float *__restrict__ d_weight) {
    __shared__ __align__(16) float sums[64][64];
    const int tid = threadIdx.x, slice = tid >> 4, at = blockIdx.x * 256 + (tid & 15) * 16;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (at < 4 * H) {
#pragma unroll 8
        for (int p = slice; p < parts; p += 64) {
            const u32x4 v = *reinterpret_cast<const u32x4 *>(partial + (int64_t)p * (4 * H) + at);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] += __uint_as_float(v[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[slice][(tid & 15) * 4 + e] = s[e];
    __syncthreads();
    const int h = blockIdx.x * 64 + tid;
    if (tid >= 64 || h >= H) return;
    float all = sums[0][tid];
    for (int k = 1; k < 64; ++k) all += sums[k][tid];
    d_weight[h] = all;
}

// How rows of nvec vectors are split: VPL vectors a lane, `waves` waves a row, `parts` rows at a time.
struct Shape {
    int vpl, waves, grid, threads;
};

Shape row_shape(int64_t parts, int nvec) {
    Shape s;
    s.vpl = nvec <= 64 ? 1 : nvec <= 1024 ? 2 : 4;
    s.waves = row_waves(nvec << 3);
    s.grid = (int)(s.waves == 1 ? (parts + kRowsAlone - 1) / kRowsAlone : parts);
    s.threads = 64 * (s.waves == 1 ? kRowsAlone : s.waves);
    return s;
}

struct NormArgs {
    const uint8_t *x;
    int64_t x_stride;
    const uint8_t *residual;
    int64_t residual_stride;
    const uint8_t *weight;
    float eps;
    int64_t rows;
    int nvec;
    uint8_t *sum;
    int64_t sum_stride;
    uint8_t *out, *codes;
    float *scales;
    hipStream_t stream;
};

template <int QUANT, int WTYPE>
void norm(const NormArgs &p) {
    const Shape s = row_shape(p.rows, p.nvec);
    auto *kernel = s.vpl == 1   ? rms_norm_kernel<1, QUANT, WTYPE>
                   : s.vpl == 2 ? rms_norm_kernel<2, QUANT, WTYPE>
                                : rms_norm_kernel<4, QUANT, WTYPE>;
    hipLaunchKernelGGL(kernel, dim3(s.grid), dim3(s.threads), 0, p.stream, p.x, p.x_stride, p.residual,
                       p.residual_stride, p.weight, p.eps, p.rows, p.nvec, s.waves, p.sum, p.sum_stride, p.out, p.codes, p.scales);
}

}  // namespace

hipError_t launch_rms_norm(const void *x, int64_t x_stride_bytes, const void *residual,
                           int64_t residual_stride_bytes, const void *weight, int32_t weight_type,
                           float eps, int64_t rows, int32_t H, int32_t quant, void *sum,
                           int64_t sum_stride_bytes, void *out, void *codes, float *scales,
                           hipStream_t stream) {
    if (rows == 0) return hipSuccess;
    const NormArgs p = {static_cast<const uint8_t *>(x), x_stride_bytes, static_cast<const uint8_t *>(residual),
                        residual_stride_bytes, static_cast<const uint8_t *>(weight), eps, rows, H / 8,
                        static_cast<uint8_t *>(sum), sum_stride_bytes, static_cast<uint8_t *>(out),
                        static_cast<uint8_t *>(codes), scales, stream};
    const bool wide = weight_type == MOE_FP32;
    if (quant == MOE_QUANT_NONE) wide ? norm<MOE_QUANT_NONE, MOE_FP32>(p) : norm<MOE_QUANT_NONE, MOE_BF16>(p);
    else if (quant == MOE_QUANT_INT8_DYN) wide ? norm<MOE_QUANT_INT8_DYN, MOE_FP32>(p) : norm<MOE_QUANT_INT8_DYN, MOE_BF16>(p);
    else wide ? norm<MOE_QUANT_FP8_E4M3_DYN, MOE_FP32>(p) : norm<MOE_QUANT_FP8_E4M3_DYN, MOE_BF16>(p);
    return hipGetLastError();
}

hipError_t launch_rms_norm_backward(const void *dy, int64_t dy_stride_bytes, const void *sum,
                                    int64_t sum_stride_bytes, const void *weight,
                                    int32_t weight_type, float eps, const void *d_sum,
                                    int64_t d_sum_stride_bytes, int64_t rows, int32_t H, void *dx,
                                    float *d_weight, void *workspace, hipStream_t stream) {
    const int nvec = H / 8, parts = (int)norm_parts(rows, H);
    if (rows > 0) {
        const Shape s = row_shape(parts, nvec);
        const auto pick = [&](auto type) {
            constexpr int T = decltype(type)::value;
            return s.vpl == 1   ? rms_norm_backward_kernel<1, T>
                   : s.vpl == 2 ? rms_norm_backward_kernel<2, T>
                                : rms_norm_backward_kernel<4, T>;
        };
        auto *kernel = weight_type == MOE_FP32 ? pick(std::integral_constant<int, MOE_FP32>{}) : pick(std::integral_constant<int, MOE_BF16>{});
        hipLaunchKernelGGL(kernel, dim3(s.grid), dim3(s.threads), 0, stream, static_cast<const uint8_t *>(dy), dy_stride_bytes,
                           static_cast<const uint8_t *>(sum), sum_stride_bytes, static_cast<const uint8_t *>(weight), eps,
                           static_cast<const uint8_t *>(d_sum), d_sum_stride_bytes, rows, nvec, s.waves,
                           static_cast<uint8_t *>(dx), parts == 1 ? reinterpret_cast<uint8_t *>(d_weight) : static_cast<uint8_t *>(workspace));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || parts == 1) return e;
    }
    hipLaunchKernelGGL(norm_weight_kernel, dim3((H + 63) / 64), dim3(1024), 0, stream,
                       static_cast<const uint8_t *>(workspace), parts, H, d_weight);
    return hipGetLastError();
}

}  // namespace moe
