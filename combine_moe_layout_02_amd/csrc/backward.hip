// The gradients of the combine and the dispatch, and the combine that keeps its rows in 8 bits, for gfx950.
//
// With y[t] = sum_k w[t,k] * row(s), s = slot_idx[t,k], and a gradient g = dy[t]:
//   d row(s) = w[t,k] * g      and      d w[t,k] = <g, row(s)>,
// so one pass over a token's K rows reads them once (bf16, or E4M3 blocks kept by the forward) and writes
// K gradient rows. The dispatch copies x[t] to K rows, so its gradient is their sum.
//
// All of it is HBM traffic with a few operations a value, and the order of the rows costs 14 to 17%: S = 4096, H =
// 7168, K = 8, rows in the layout's order and in token order: the combine's gradient 199 and 170 us (998 MB), from a
// checkpoint 161 and 144, the checkpointed combine 146 and 128. The scattered reads alone cost less: the combine reads the
// same rows in 84 us, 77 in token order, and the planned pack, which writes such rows in slot order, takes
// 84 too, so what is lost here is lost by token-order writes among the reads. A pass that only reads and a second that
// writes in slot order from the layout's records have not been tried. Two ways to do both in slot order, through an inverse
// of slot_idx that a first kernel writes, came to 196 us (a workgroup a row) and 205 us (a workgroup a quarter row, sums
// joined by a third kernel) where this kernel took 213: the gain is spent on the second read of dy for every row, the
// chain from slot to token to dy, and the launches; a call would need a workspace too.
//
// Below that size occupancy and the last round of workgroups count: 1531 tokens of 2080, K = 6, move their 62 MB at 3.5
// to 3.7 TB/s. combine_backward_kernel holds a slot and descriptors for every row in scalar registers, of which some
// spill to vector lanes (bf16 rows and a checkpoint's: 24 and 72 with KMAX = 8, 210 and 346 with 16); with KMAX = 4
// on bf16 rows the compiler keeps a small array in 16 KB of LDS, so nine waves fit a compute unit where rows are short
// (8192 tokens of 512, K = 4: 27.6 us, its bytes 11.4).

#include "mx_blocks.h"

namespace moe {
namespace {

using namespace mx;

constexpr int kLoadPolicy = 2;              // nt: rows are read once
constexpr int kStorePolicy = 1 | 16;        // sc0 sc1
constexpr int kStreamPolicy = 1 | 16 | 2;   // sc0 sc1 nt: a checkpoint's codes stream to HBM
// nt: gradient rows, chosen with the calls that follow in the stream (S = 4096, H = 7168, K = 8, us with nt, kStreamPolicy
// and write-back): the gradient alone 199.9, 201.7 and 206.8, with the dispatch's gradient of the rows behind it 286.2,
// 286.2 and 270.3, with a copy of 400 MB 361.3, 361.5 and 361.8; from a checkpoint 161.1, 162.4 and 171.6, between the
// checkpointed combine and the dispatch's gradient 392.8, 393.0 and 395.7, before the copy 325.4, 325.4 and 336.2.
constexpr int kRowPolicy = 2;
// A checkpoint's values are taken at half their size, and the sums doubled: a block's largest can be 2^128, past
// fp32, whose product with a small or zero gradient is finite.
constexpr float kHalf = 0.5f;
// 16-byte vectors of a part, a lane each. S = 4096, H = 7168, K = 8: the dispatch's gradient takes 84.5 us with
// 32, 86.0 with 64 and 85.9 with 128; the checkpointed combine 159, 146 and 146 (a row's codes are half as wide).
template <bool KEEP>
constexpr int part_threads() { return KEEP ? 64 : 32; }

__device__ inline __amdgpu_buffer_rsrc_t rsrc(const void *base, int32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, bytes, 0x00020000);
}

// Sum over the 64 lanes of a wave of each of N values (N a power of two up to 16); afterwards lane l holds the
// sum of value l * N / 64, in a fixed order. Each step halves the values a lane carries and swaps the
// other half with the lane across.
template <int N>
__device__ inline float wave_sums(float (&v)[N]) {
    const int lane = threadIdx.x & 63;
    int d = 32;
#pragma unroll
    for (int n = N; n > 1; n >>= 1, d >>= 1) {
        const bool up = lane & d;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float send = up ? v[i] : v[i + n / 2];
            const float keep = up ? v[i + n / 2] : v[i];
            v[i] = keep + __shfl_xor(send, d, 64);
        }
    }
    float s = v[0];
    for (; d > 0; d >>= 1) s += __shfl_xor(s, d, 64);
    return s;
}

// grid = S; workgroup t takes token t, its lanes vectors threadIdx.x, + blockDim.x, ... of the rows (at most two
// rounds: nvec <= 2048 and 1024 lanes; a lane a vector where they suffice, so that all of a token's loads are
// under way at once. S = 4096, K = 8, this, 64 lanes with more rounds and 256: 199, 198 and 200 us at H = 7168, 111, 123 and
// 110 at 4096, 57, 67 and 57 at 2048; 8192 tokens of 4096 219, 258 and 225; 64 tokens of 7168 9.2, 21.6 and 10.4). An eighth
// of the tokens in order for each XCD takes 199, 114 and 57 us at those H, and 225 with 8192 tokens.
// MX: the rows are E4M3 codes and scales (stride = H). d_weights: a lane's sum over its values in order, the wave's
// lanes by a fixed tree, the waves in order, all in fp32.
template <int KMAX, bool MX>
__global__ __launch_bounds__(1024) void combine_backward_kernel(
    const uint8_t *__restrict__ dy, const uint8_t *__restrict__ rows, const uint8_t *__restrict__ scales,
    int64_t stride, int64_t nrows, const int32_t *__restrict__ slot_idx,
    const float *__restrict__ weights, int K, int nvec, uint8_t *__restrict__ d_rows,
    int64_t d_stride, float *__restrict__ d_weights) {
    __shared__ float partial[16][KMAX];
    const int64_t t = blockIdx.x;
    const int row_bytes = nvec << 4;
    int64_t slot[KMAX];
    float w[KMAX], sum[KMAX];
#pragma unroll
    for (int k = 0; k < KMAX; ++k) {
        const int64_t s = k < K ? slot_idx[t * K + k] : -1;
        slot[k] = s >= 0 && s < nrows ? s : -1;
        w[k] = slot[k] >= 0 ? weights[t * K + k] : 0.0f;
        sum[k] = 0.0f;
    }
    const __amdgpu_buffer_rsrc_t g_src = rsrc(dy + t * row_bytes, row_bytes);
    for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
        const u32x4 g = __builtin_amdgcn_raw_buffer_load_b128(g_src, v << 4, 0, kLoadPolicy);
        u32x4 x[KMAX];
        uint32_t byte[KMAX];
#pragma unroll
        for (int k = 0; k < KMAX; ++k) {
            if (slot[k] < 0) continue;
            if constexpr (MX) {
                const u32x2 c = __builtin_amdgcn_raw_buffer_load_b64(
                    rsrc(rows + slot[k] * stride, nvec << 3), v << 3, 0, kLoadPolicy);
                x[k] = u32x4{c.x, c.y, 0u, 0u};
                byte[k] = __builtin_amdgcn_raw_buffer_load_b8(
                    rsrc(scales + slot[k] * (nvec >> 2), nvec >> 2), v >> 2, 0, 0);
            } else {
                x[k] = __builtin_amdgcn_raw_buffer_load_b128(rsrc(rows + slot[k] * stride, row_bytes),
                                                             v << 4, 0, kLoadPolicy);
            }
        }
        float gf[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            gf[2 * i] = bf16_lo(g[i]);
            gf[2 * i + 1] = bf16_hi(g[i]);
        }
#pragma unroll
        for (int k = 0; k < KMAX; ++k) {
            if (slot[k] < 0) continue;
            float xf[8];
            if constexpr (MX) {
                decode_e4m3(u32x2{x[k][0], x[k][1]}, kHalf * scale_value(byte[k]), xf);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    xf[2 * i] = bf16_lo(x[k][i]);
                    xf[2 * i + 1] = bf16_hi(x[k][i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[k] = __builtin_fmaf(gf[i], xf[i], sum[k]);
            u32x4 out;
#pragma unroll
            for (int i = 0; i < 4; ++i) out[i] = bf16_pair(w[k] * gf[2 * i], w[k] * gf[2 * i + 1]);
            __builtin_amdgcn_raw_buffer_store_b128(out, rsrc(d_rows + slot[k] * d_stride, row_bytes),
                                                   v << 4, 0, kRowPolicy);
        }
    }
    const float s = wave_sums<KMAX>(sum);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (lane % (64 / KMAX) == 0) partial[wave][lane / (64 / KMAX)] = s;
    __syncthreads();
    if (threadIdx.x < K) {
        float total = 0.0f;
        const int nwaves = (blockDim.x + 63) >> 6;
        for (int i = 0; i < nwaves; ++i) total += partial[i][threadIdx.x];
        const int64_t sk = slot_idx[t * K + threadIdx.x];
        d_weights[t * K + threadIdx.x] = sk >= 0 && sk < nrows ? total * (MX ? 1.0f / kHalf : 1.0f) : 0.0f;
    }
}

// The dispatch's gradient, and the combine that keeps its rows. Parts and their order as in the combine: grid
// = 8 * ceil(S / 8) * nparts, all parts of token t on XCD t % 8.
//   KEEP = false: dx[t] = sum of the token's rows.
//   KEEP = true:  y[t] = the weighted sum, each product and each sum rounded to fp32 on its own as in the
//                 combine (this file is compiled with -ffp-contract=off), and the rows' E4M3 blocks.
template <int KMAX, bool KEEP>
__global__ __launch_bounds__(part_threads<KEEP>()) void gather_kernel(
    const uint8_t *__restrict__ rows, int64_t stride, int64_t nrows,
    const int32_t *__restrict__ slot_idx, const float *__restrict__ weights, int S, int K, int nvec,
    int nparts, uint8_t *__restrict__ out, uint8_t *__restrict__ codes,
    uint8_t *__restrict__ scales) {
    const int m = blockIdx.x >> 3;
    const int i = m / nparts;
    const int q = m - i * nparts;
    const int64_t t = 8 * i + (blockIdx.x & 7);
    if (t >= S) return;
    const int v = q * part_threads<KEEP>() + threadIdx.x;
    const int row_bytes = nvec << 4;
    int64_t slot[KMAX];
    float w[KMAX];
#pragma unroll
    for (int k = 0; k < KMAX; ++k) {
        const int64_t s = k < K ? slot_idx[t * K + k] : -1;
        slot[k] = s >= 0 && s < nrows ? s : -1;
        w[k] = KEEP && slot[k] >= 0 ? weights[t * K + k] : 1.0f;
    }
    if (v >= nvec) return;  // with KEEP nvec is a multiple of 4: a block's lanes leave or stay together
    u32x4 x[KMAX];
#pragma unroll
    for (int k = 0; k < KMAX; ++k)
        if (slot[k] >= 0)
            x[k] = __builtin_amdgcn_raw_buffer_load_b128(rsrc(rows + slot[k] * stride, row_bytes), v << 4, 0,
                                                         kLoadPolicy);
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
#pragma unroll
    for (int k = 0; k < KMAX; ++k) {
        if (slot[k] < 0) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float lo = bf16_lo(x[k][e]), hi = bf16_hi(x[k][e]);
            acc[2 * e] = acc[2 * e] + (KEEP ? w[k] * lo : lo);
            acc[2 * e + 1] = acc[2 * e + 1] + (KEEP ? w[k] * hi : hi);
        }
        if constexpr (KEEP) {
            const uint32_t byte = scale_byte<MOE_MX_E4M3>(max_of_four_lanes(amax_bits(x[k])));
            const u32x2 c = encode<MOE_MX_E4M3>(x[k], byte);
            __builtin_amdgcn_raw_buffer_store_b64(
                c, rsrc(codes + slot[k] * (int64_t)(nvec << 3), nvec << 3), v << 3, 0, kStreamPolicy);
            if ((threadIdx.x & 3) == 0)
                scales[slot[k] * (int64_t)(nvec >> 2) + (v >> 2)] = (uint8_t)byte;
        }
    }
    u32x4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = bf16_pair(acc[2 * e], acc[2 * e + 1]);
    __builtin_amdgcn_raw_buffer_store_b128(r, rsrc(out + t * row_bytes, row_bytes), v << 4, 0,
                                           kStorePolicy);
}

template <int KMAX, bool MX>
hipError_t backward(const void *dy, const void *rows, const void *scales, int64_t stride, int64_t nrows,
                    const int32_t *slot_idx, const float *weights, int S, int H, int K, void *d_rows,
                    int64_t d_stride, float *d_weights, hipStream_t stream) {
    const int nvec = H / 8;
    const int threads = nvec >= 1024 ? 1024 : (nvec + 63) / 64 * 64;
    hipLaunchKernelGGL((combine_backward_kernel<KMAX, MX>), dim3(S), dim3(threads), 0, stream,
                       static_cast<const uint8_t *>(dy), static_cast<const uint8_t *>(rows),
                       static_cast<const uint8_t *>(scales), stride, nrows, slot_idx, weights, K, nvec,
                       static_cast<uint8_t *>(d_rows), d_stride, d_weights);
    return hipGetLastError();
}

template <bool MX>
hipError_t backward_k(const void *dy, const void *rows, const void *scales, int64_t stride, int64_t nrows,
                      const int32_t *slot_idx, const float *weights, int S, int H, int K, void *d_rows,
                      int64_t d_stride, float *d_weights, hipStream_t stream) {
    if (K <= 2)
        return backward<2, MX>(dy, rows, scales, stride, nrows, slot_idx, weights, S, H, K, d_rows, d_stride, d_weights, stream);
    if (K <= 4)
        return backward<4, MX>(dy, rows, scales, stride, nrows, slot_idx, weights, S, H, K, d_rows, d_stride, d_weights, stream);
    if (K <= 8)
        return backward<8, MX>(dy, rows, scales, stride, nrows, slot_idx, weights, S, H, K, d_rows, d_stride, d_weights, stream);
    return backward<16, MX>(dy, rows, scales, stride, nrows, slot_idx, weights, S, H, K, d_rows, d_stride, d_weights, stream);
}

template <int KMAX, bool KEEP>
hipError_t gather(const void *rows, int64_t stride, int64_t nrows, const int32_t *slot_idx,
                  const float *weights, int S, int H, int K, void *out, void *codes, void *scales,
                  hipStream_t stream) {
    const int nvec = H / 8;
    constexpr int lanes = part_threads<KEEP>();
    const int nparts = (nvec + lanes - 1) / lanes;
    const uint32_t grid = 8u * (uint32_t)((S + 7) / 8) * (uint32_t)nparts;
    hipLaunchKernelGGL((gather_kernel<KMAX, KEEP>), dim3(grid), dim3(lanes), 0, stream,
                       static_cast<const uint8_t *>(rows), stride, nrows, slot_idx, weights, S, K, nvec,
                       nparts, static_cast<uint8_t *>(out), static_cast<uint8_t *>(codes),
                       static_cast<uint8_t *>(scales));
    return hipGetLastError();
}

template <bool KEEP>
hipError_t gather_k(const void *rows, int64_t stride, int64_t nrows, const int32_t *slot_idx,
                    const float *weights, int S, int H, int K, void *out, void *codes, void *scales,
                    hipStream_t stream) {
    if (K <= 2) return gather<2, KEEP>(rows, stride, nrows, slot_idx, weights, S, H, K, out, codes, scales, stream);
    if (K <= 4) return gather<4, KEEP>(rows, stride, nrows, slot_idx, weights, S, H, K, out, codes, scales, stream);
    if (K <= 8) return gather<8, KEEP>(rows, stride, nrows, slot_idx, weights, S, H, K, out, codes, scales, stream);
    return gather<16, KEEP>(rows, stride, nrows, slot_idx, weights, S, H, K, out, codes, scales, stream);
}

}  // namespace

hipError_t launch_combine_backward(const void *dy, const void *expert_out, int64_t row_stride_bytes,
                                   int64_t expert_rows, const int32_t *slot_idx,
                                   const float *topk_weights, int32_t S, int32_t H, int32_t K,
                                   void *d_expert_out, int64_t d_row_stride_bytes,
                                   float *d_topk_weights, hipStream_t stream) {
    return backward_k<false>(dy, expert_out, nullptr, row_stride_bytes, expert_rows, slot_idx,
                             topk_weights, S, H, K, d_expert_out, d_row_stride_bytes, d_topk_weights,
                             stream);
}

hipError_t launch_combine_backward_mx(const void *dy, const void *codes, const void *scales,
                                      int64_t expert_rows, const int32_t *slot_idx,
                                      const float *topk_weights, int32_t S, int32_t H, int32_t K,
                                      void *d_expert_out, int64_t d_row_stride_bytes,
                                      float *d_topk_weights, hipStream_t stream) {
    return backward_k<true>(dy, codes, scales, H, expert_rows, slot_idx, topk_weights, S, H, K,
                            d_expert_out, d_row_stride_bytes, d_topk_weights, stream);
}

hipError_t launch_dispatch_backward(const void *d_rows, int64_t row_stride_bytes,
                                    int64_t expert_rows, const int32_t *slot_idx, int32_t S,
                                    int32_t H, int32_t K, void *dx, hipStream_t stream) {
    return gather_k<false>(d_rows, row_stride_bytes, expert_rows, slot_idx, nullptr, S, H, K, dx,
                           nullptr, nullptr, stream);
}

hipError_t launch_combine_checkpoint(const void *expert_out, int64_t row_stride_bytes,
                                     int64_t expert_rows, const int32_t *slot_idx,
                                     const float *topk_weights, int32_t S, int32_t H, int32_t K,
                                     void *y, void *codes, void *scales, hipStream_t stream) {
    return gather_k<true>(expert_out, row_stride_bytes, expert_rows, slot_idx, topk_weights, S, H, K,
                          y, codes, scales, stream);
}

}  // namespace moe
