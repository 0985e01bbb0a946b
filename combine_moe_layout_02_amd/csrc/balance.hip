// The router's balance loss over the experts' counts, and its gradient, for gfx950 (see moe_balance_loss in moe.h).
//
// A wave takes a token: lane l holds experts l, l + 64, ... of it, so that its scores are two reductions over the wave's
// lanes, and their sums over tokens stay in its registers. All of it is a few bytes and operations a logit.

#include "moe_internal.h"

namespace moe {
namespace {

typedef __bf16 bf16_t;

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kFinishThreads = 1024;

__device__ inline float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

__device__ inline int wave_sum(int v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

__device__ inline float wave_max(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
    return v;
}

// The scores of one token from its logits (-inf past E): exp(l - max) over their sum, or sigmoids over theirs. Those are
// taken as exp(min(l, 0) - min(max, 0)) / (1 + exp(-|l|)), sigmoid(l) but for one factor, so that a token whose
// logits are all far below zero keeps its scores. With no logit above -inf there are none.
template <int N, int SCORE>
__device__ inline void scores_of(const float (&l)[N], float (&s)[N]) {
    float top = l[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, l[i]);
    top = wave_max(top);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        s[i] = SCORE == MOE_SCORE_SIGMOID ? expf(fminf(l[i], 0.0f) - fminf(top, 0.0f)) / (1.0f + expf(-fabsf(l[i])))
                                          : expf(l[i] - top);
        sum += s[i];
    }
    sum = wave_sum(sum);
    const bool none = top == -__builtin_inff();
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = none ? 0.0f : s[i] / sum;
}

template <int N, class T>
__device__ inline void load_logits(const uint8_t *__restrict__ row, int E, float (&l)[N]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = lane + 64 * i;
        l[i] = e < E ? (float)reinterpret_cast<const T *>(row)[e] : -__builtin_inff();
    }
}

// loss from the counts and the sums of scores; n entries and tokens in all. Every lane of a wave calls this with its
// share of sum over e of count * score sum.
__device__ inline float loss_of(double share, int64_t n, int tokens, int E, float coef) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) share += __shfl_xor(share, d, 64);
    return tokens ? (float)(share * ((double)coef * E / ((double)n * tokens))) : 0.0f;
}

// Part p takes tokens [p * per, ...), its waves every fourth of them. A single part finishes by itself; several leave
// their sums, counts and tokens in the workspace.
template <int N, int SCORE, class T>
__global__ __launch_bounds__(kThreads) void balance_parts_kernel(
    const uint8_t *__restrict__ logits, int64_t stride, const int32_t *__restrict__ topk, int S, int K, int E,
    int per, float coef, float *__restrict__ loss, int32_t *__restrict__ counts, int32_t *__restrict__ tokens,
    float *__restrict__ part_sums, int32_t *__restrict__ part_counts, int32_t *__restrict__ part_tokens) {
    __shared__ int32_t count[MOE_MAX_EXPERTS];
    __shared__ float sums[kWaves][MOE_MAX_EXPERTS];
    __shared__ int32_t live[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < E; e += kThreads) count[e] = 0;
    __syncthreads();
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    int lives = 0;
    const int end = min(S, (int)(blockIdx.x + 1) * per);
    for (int t = blockIdx.x * per + wave; t < end; t += kWaves) {
        float l[N], s[N];
        load_logits<N, T>(logits + t * stride, E, l);
        const int e = lane < K ? topk[(int64_t)t * K + lane] : -1;
        const bool valid = e >= 0 && e < E;
        if (valid) atomicAdd(&count[e], 1);
        if (!__any(valid)) continue;
        ++lives;
        scores_of<N, SCORE>(l, s);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += s[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (lane + 64 * i < E) sums[wave][lane + 64 * i] = acc[i];
    if (lane == 0) live[wave] = lives;
    __syncthreads();
    int all = 0;
    for (int w = 0; w < kWaves; ++w) all += live[w];
    if (gridDim.x > 1) {
        for (int e = tid; e < E; e += kThreads) {
            float s = sums[0][e];
            for (int w = 1; w < kWaves; ++w) s += sums[w][e];
            part_sums[(int64_t)blockIdx.x * E + e] = s;
            part_counts[(int64_t)blockIdx.x * E + e] = count[e];
        }
        if (tid == 0) part_tokens[blockIdx.x] = all;
        return;
    }
    if (wave > 0) return;
    double share = 0.0;
    int n = 0;
    for (int e = lane; e < E; e += 64) {
        float s = sums[0][e];
        for (int w = 1; w < kWaves; ++w) s += sums[w][e];
        share += (double)count[e] * (double)s;
        n += count[e];
        counts[e] = count[e];
    }
    const float value = loss_of(share, wave_sum(n), all, E, coef);
    if (lane == 0) *loss = value, *tokens = all;
}

// One workgroup: expert e = tid % width, slice tid / width of the parts (width = E rounded up to a power of two), then the
// slices in order.
__global__ __launch_bounds__(kFinishThreads) void balance_finish_kernel(
    const float *__restrict__ part_sums, const int32_t *__restrict__ part_counts,
    const int32_t *__restrict__ part_tokens, int parts, int E, int width, float coef, float *__restrict__ loss,
    int32_t *__restrict__ counts, int32_t *__restrict__ tokens) {
    __shared__ float sums[kFinishThreads];
    __shared__ int32_t count[kFinishThreads];
    const int tid = threadIdx.x, e = tid & (width - 1), slice = tid / width, slices = kFinishThreads / width;
    float s = 0.0f;
    int c = 0;
    if (e < E)
        for (int p = slice; p < parts; p += slices) {
            s += part_sums[(int64_t)p * E + e];
            c += part_counts[(int64_t)p * E + e];
        }
    sums[tid] = s;
    count[tid] = c;
    __syncthreads();
    if (tid >= 64) return;
    double share = 0.0;
    int n = 0, lives = 0;
    for (int at = tid; at < E; at += 64) {
        float sum = 0.0f;
        int all = 0;
        for (int k = 0; k < slices; ++k) {
            sum += sums[k * width + at];
            all += count[k * width + at];
        }
        share += (double)all * (double)sum;
        n += all;
        counts[at] = all;
    }
    for (int p = tid; p < parts; p += 64) lives += part_tokens[p];
    lives = wave_sum(lives);
    const float value = loss_of(share, wave_sum(n), lives, E, coef);
    if (tid == 0) *loss = value, *tokens = lives;
}

// A wave a token, as above. n[e] counts from the mean, which takes nothing from the gradient (the scores' sum is 1), and
// lets equal counts cancel exactly.
template <int N, int SCORE, class T>
__global__ __launch_bounds__(kThreads) void balance_backward_kernel(
    const float *__restrict__ d_loss, const uint8_t *__restrict__ logits, int64_t stride,
    const int32_t *__restrict__ topk, const int32_t *__restrict__ counts, const int32_t *__restrict__ tokens, int S,
    int K, int E, float coef, T *__restrict__ d_logits) {
    const int lane = threadIdx.x & 63, step = gridDim.x * kWaves;
    int n[N], sum = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        n[i] = lane + 64 * i < E ? counts[lane + 64 * i] : 0;
        sum += n[i];
    }
    sum = wave_sum(sum);
    const int mean = sum / E;
    const double all = (double)sum * (double)*tokens;
    const float each = all > 0.0 ? (float)((double)coef * E / all) * *d_loss : 0.0f;
    for (int t = blockIdx.x * kWaves + (threadIdx.x >> 6); t < S; t += step) {
        float l[N], s[N], g[N];
        load_logits<N, T>(logits + t * stride, E, l);
        const int id = lane < K ? topk[(int64_t)t * K + lane] : -1;
        const bool lives = __any(id >= 0 && id < E);
        scores_of<N, SCORE>(l, s);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            g[i] = (float)(n[i] - mean);
            dot += lane + 64 * i < E ? g[i] * s[i] : 0.0f;
        }
        dot = wave_sum(dot);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = lane + 64 * i;
            if (e >= E) continue;
            float d = each * (s[i] * (g[i] - dot));
            if (SCORE == MOE_SCORE_SIGMOID) {
                const float far = expf(-fabsf(l[i]));
                d *= (l[i] > 0.0f ? far : 1.0f) / (1.0f + far);
            }
            d_logits[(int64_t)t * E + e] = (T)(lives ? d : 0.0f);
        }
    }
}

// The kernel of the call's sizes and types: f(N lanes' experts, score, element) for constants of each.
template <class F>
void dispatch(int32_t E, int32_t type, int32_t score, F f) {
    const auto typed = [&](auto n, auto s) {
        if (type == MOE_BF16) f(n, s, bf16_t{});
        else f(n, s, float{});
    };
    const auto scored = [&](auto n) {
        if (score == MOE_SCORE_SIGMOID) typed(n, std::integral_constant<int, MOE_SCORE_SIGMOID>{});
        else typed(n, std::integral_constant<int, MOE_SCORE_SOFTMAX>{});
    };
    if (E <= 64) scored(std::integral_constant<int, 1>{});
    else if (E <= 128) scored(std::integral_constant<int, 2>{});
    else if (E <= 256) scored(std::integral_constant<int, 4>{});
    else scored(std::integral_constant<int, 8>{});
}

}  // namespace

hipError_t launch_balance_loss(const void *logits, int64_t logits_stride_bytes, int32_t logits_type,
                               const int32_t *topk_idx, int32_t S, int32_t K, int32_t E,
                               int32_t score, float coef, float *loss,
                               int32_t *num_tokens_per_expert, int32_t *num_tokens, void *workspace,
                               hipStream_t stream) {
    const int most = balance_parts(S), per = (S + most - 1) / most, parts = (S + per - 1) / per;
    float *sums = static_cast<float *>(workspace);
    int32_t *counts = parts > 1 ? reinterpret_cast<int32_t *>(sums + (int64_t)parts * E) : nullptr;
    int32_t *tokens = parts > 1 ? counts + (int64_t)parts * E : nullptr;
    dispatch(E, logits_type, score, [&](auto n, auto s, auto element) {
        hipLaunchKernelGGL((balance_parts_kernel<decltype(n)::value, decltype(s)::value, decltype(element)>), dim3(parts),
                           dim3(kThreads), 0, stream, static_cast<const uint8_t *>(logits), logits_stride_bytes, topk_idx,
                           S, K, E, per, coef, loss, num_tokens_per_expert, num_tokens, sums, counts, tokens);
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || parts == 1) return e;
    int width = 1;
    while (width < E) width *= 2;
    hipLaunchKernelGGL(balance_finish_kernel, dim3(1), dim3(kFinishThreads), 0, stream, sums, counts, tokens, parts, E,
                       width, coef, loss, num_tokens_per_expert, num_tokens);
    return hipGetLastError();
}

hipError_t launch_balance_loss_backward(const float *d_loss, const void *logits,
                                        int64_t logits_stride_bytes, int32_t logits_type,
                                        const int32_t *topk_idx,
                                        const int32_t *num_tokens_per_expert,
                                        const int32_t *num_tokens, int32_t S, int32_t K, int32_t E,
                                        int32_t score, float coef, void *d_logits,
                                        hipStream_t stream) {
    const int need = (S + kWaves - 1) / kWaves, grid = need < 2048 ? need : 2048;
    dispatch(E, logits_type, score, [&](auto n, auto s, auto element) {
        using T = decltype(element);
        hipLaunchKernelGGL((balance_backward_kernel<decltype(n)::value, decltype(s)::value, T>), dim3(grid), dim3(kThreads),
                           0, stream, d_loss, static_cast<const uint8_t *>(logits), logits_stride_bytes, topk_idx,
                           num_tokens_per_expert, num_tokens, S, K, E, coef, static_cast<T *>(d_logits));
    });
    return hipGetLastError();
}

}  // namespace moe
