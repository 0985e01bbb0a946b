// The router's balance loss over the experts' counts, and its gradient, for gfx950 (see moe_balance_loss in moe.h).
//
// A wave takes a token: lane l holds experts l, l + 64, ... of it, so that its scores are two reductions over the wave's
// lanes, and their sums over tokens stay in its registers. The exponentials and the reductions' chains bound it, and launches:
// 8192 tokens of 256 experts (8.4 MB) take 12.9 us forward, 6.0 in the parts and 7 in the one workgroup that joins 256 of
// them, and 6.5 back, 128 tokens of 16 experts (one part) 7.4 and 4.6. Parts of 128 tokens (64 of them) took 20 + 4.6, of 64
// 8.0 + 6.4; with the library's expf, divisions and shuffles 13.6 + 20. The gradient with 1024 workgroups the same, 512
// 7.4, 256 10.8.

#include "wave_ops.h"

namespace moe {
namespace {

typedef __bf16 bf16_t;

constexpr int kPartThreads = 1024, kPartWaves = kPartThreads / 64;
constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kFinishThreads = 1024;
constexpr int kFinishSlices = 32;
constexpr int kBackwardGrid = 2048;

// exp(x) for x <= 0 to 2 ulp, from the hardware's exp2 of x * log2(e) and the rest of that product; 0 from -200 down, NaN of a
// NaN. A third of the library function's instructions, which bound these kernels.
__device__ inline float exp_of(float x) {
    constexpr float kLog2e = 1.44269502e+00f, kLog2eRest = 1.92596299e-08f, kLn2 = 6.93147182e-01f;
    x = x < -200.0f ? -200.0f : x;
    const float t = x * kLog2e;
    const float rest = __builtin_fmaf(x, kLog2eRest, __builtin_fmaf(x, kLog2e, -t));
    const float y = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(y, rest * kLn2, y);
}

// The scores of one token from its logits (-inf past E): exp(l - max) over their sum, or sigmoids over theirs. A token whose
// logits are all far below zero, where sigmoid(l) is exp(l) to fp32, keeps its scores: they are taken against the
// largest. A logit of -inf has score 0, also where there is no other. turn: 1 - sigmoid(l), for MOE_SCORE_SIGMOID.
template <int N, int SCORE>
__device__ inline void scores_of(const float (&l)[N], float (&s)[N], float (&turn)[N]) {
    float top = l[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, l[i]);
    top = wave::most(top);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (SCORE == MOE_SCORE_SIGMOID) {
            const float far = exp_of(-fabsf(l[i])), share = __builtin_amdgcn_rcpf(1.0f + far);
            turn[i] = (l[i] > 0.0f ? far : 1.0f) * share;
            s[i] = top < -60.0f ? exp_of(l[i] - top) : (l[i] > 0.0f ? 1.0f : far) * share;
        } else {
            s[i] = exp_of(l[i] - top);
        }
        sum += s[i];
    }
    const float each = 1.0f / wave::sum(sum);
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = l[i] == -__builtin_inff() ? 0.0f : s[i] * each;
}

// A token's logits (-inf past E) and entries (-1 past K) in a wave's lanes; nothing of tokens past the end.
template <int N, class T>
struct Token {
    float l[N];
    int id;
    __device__ void load(const uint8_t *__restrict__ logits, int64_t stride, const int32_t *__restrict__ topk, int t, int end, int K, int E) {
        const int lane = threadIdx.x & 63;
        const T *row = reinterpret_cast<const T *>(logits + t * stride);
#pragma unroll
        for (int i = 0; i < N; ++i) l[i] = t < end && lane + 64 * i < E ? (float)row[lane + 64 * i] : -__builtin_inff();
        id = t < end && lane < K ? topk[(int64_t)t * K + lane] : -1;
    }
};

// The loss from sum over e of count * score sum, of n entries and tokens in all.
__device__ inline float loss_of(double share, int64_t n, int tokens, int E, float coef) {
    return tokens ? (float)(share * ((double)coef * E / ((double)n * tokens))) : 0.0f;
}

// Part p takes tokens [p * per, ...), its waves every sixteenth of them, the next one's loads under way. A single part
// finishes by itself; several leave their sums, counts and tokens in the workspace.
template <int N, int SCORE, class T>
__global__ __launch_bounds__(kPartThreads) void balance_parts_kernel(
    const uint8_t *__restrict__ logits, int64_t stride, const int32_t *__restrict__ topk, int S, int K, int E,
    int per, float coef, float *__restrict__ loss, int32_t *__restrict__ counts, int32_t *__restrict__ tokens,
    float *__restrict__ part_sums, uint16_t *__restrict__ part_counts, int32_t *__restrict__ part_tokens) {
    __shared__ int32_t count[64 * N];
    __shared__ float sums[kPartWaves][64 * N];
    __shared__ int32_t live[kPartWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < 64 * N; e += kPartThreads) count[e] = 0;
    __syncthreads();
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    int lives = 0;
    const int end = min(S, (int)(blockIdx.x + 1) * per);
    int t = blockIdx.x * per + wave;
    Token<N, T> next;
    next.load(logits, stride, topk, t, end, K, E);
    for (; t < end; t += kPartWaves) {
        const Token<N, T> token = next;
        next.load(logits, stride, topk, t + kPartWaves, end, K, E);
        const bool valid = token.id >= 0 && token.id < E;
        if (valid) atomicAdd(&count[token.id], 1);
        if (!__any(valid)) continue;
        ++lives;
        float s[N], turn[N];
        scores_of<N, SCORE>(token.l, s, turn);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += s[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) sums[wave][lane + 64 * i] = acc[i];
    if (lane == 0) live[wave] = lives;
    __syncthreads();
    int all = 0;
    for (int w = 0; w < kPartWaves; ++w) all += live[w];
    const auto sum_of = [&](int e) {
        float s = sums[0][e];
#pragma unroll
        for (int w = 1; w < kPartWaves; ++w) s += sums[w][e];
        return s;
    };
    if (gridDim.x > 1) {
        const int wide = (E + 3) / 4 * 4;  // experts up to there have no scores and no entries
        for (int e = tid; e < wide; e += kPartThreads) {
            part_sums[blockIdx.x * wide + e] = sum_of(e);
            part_counts[blockIdx.x * wide + e] = (uint16_t)count[e];  // 256 tokens of 16 entries at most
        }
        if (tid == 0) part_tokens[blockIdx.x] = all;
        return;
    }
    if (wave > 0) return;
    double share = 0.0;
    int n = 0;
    for (int e = lane; e < E; e += 64) {
        share += (double)count[e] * (double)sum_of(e);
        n += count[e];
        counts[e] = count[e];
    }
    const float value = loss_of(wave::sum(share), wave::sum(n), all, E, coef);
    if (lane == 0) *loss = value, *tokens = all;
}

// One workgroup: four experts a thread, `groups` threads (E / 4 rounded up to a power of two) to a part's row, as many parts
// at once as there are threads for them, 32 at most; then the threads' sums in order.
__global__ __launch_bounds__(kFinishThreads) void balance_finish_kernel(
    const float *__restrict__ part_sums, const uint16_t *__restrict__ part_counts,
    const int32_t *__restrict__ part_tokens, int parts, int E, int groups, float coef, float *__restrict__ loss,
    int32_t *__restrict__ counts, int32_t *__restrict__ tokens) {
    __shared__ float sums[4 * kFinishThreads];
    __shared__ int32_t count[4 * kFinishThreads];
    __shared__ double share[kFinishThreads / 64];
    __shared__ int32_t entries[kFinishThreads / 64], lives[kFinishThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wide = (E + 3) / 4 * 4, e = (tid & (groups - 1)) * 4, slice = tid / groups, slices = min(kFinishThreads / groups, kFinishSlices);
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int c[4] = {0, 0, 0, 0}, live = 0;
    if (e < wide && slice < slices) {
#pragma unroll 16
        for (int p = slice; p < parts; p += slices) {
            const float4 f = *reinterpret_cast<const float4 *>(part_sums + p * wide + e);
            const ushort4 n = *reinterpret_cast<const ushort4 *>(part_counts + p * wide + e);
            s[0] += f.x, s[1] += f.y, s[2] += f.z, s[3] += f.w;
            c[0] += n.x, c[1] += n.y, c[2] += n.z, c[3] += n.w;
        }
    }
    if (tid < parts) live = part_tokens[tid];
    if (slice < slices) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sums[slice * 4 * groups + e + i] = s[i];
            count[slice * 4 * groups + e + i] = c[i];
        }
    }
    __syncthreads();
    double part = 0.0;
    int all = 0;
    if (tid < E) {
        float sum = 0.0f;
#pragma unroll 4
        for (int k = 0; k < slices; ++k) {
            sum += sums[k * 4 * groups + tid];
            all += count[k * 4 * groups + tid];
        }
        part = (double)all * (double)sum;
        counts[tid] = all;
    }
    part = wave::sum(part);
    all = wave::sum(all);
    live = wave::sum(live);
    if (lane == 0) share[wave] = part, entries[wave] = all, lives[wave] = live;
    __syncthreads();
    if (tid > 0) return;
    int n = 0, live_all = 0;
    part = 0.0;
    for (int w = 0; w < kFinishThreads / 64; ++w) part += share[w], n += entries[w], live_all += lives[w];
    *loss = loss_of(part, n, live_all, E, coef);
    *tokens = live_all;
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
    sum = wave::sum(sum);
    const int mean = sum / E;
    const double all = (double)sum * (double)*tokens;
    const float each = all > 0.0 ? (float)((double)coef * E / all) * *d_loss : 0.0f;
    int t = blockIdx.x * kWaves + (threadIdx.x >> 6);
    Token<N, T> next;
    next.load(logits, stride, topk, t, S, K, E);
    for (; t < S; t += step) {
        const Token<N, T> token = next;
        next.load(logits, stride, topk, t + step, S, K, E);
        const bool lives = __any(token.id >= 0 && token.id < E);
        float s[N], turn[N], g[N];
        scores_of<N, SCORE>(token.l, s, turn);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            g[i] = (float)(n[i] - mean);
            dot += g[i] * s[i];
        }
        dot = wave::sum(dot);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = lane + 64 * i;
            if (e >= E) continue;
            float d = each * (s[i] * (g[i] - dot));
            if (SCORE == MOE_SCORE_SIGMOID) d *= turn[i];
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
    const int64_t each = (int64_t)most * ((E + 3) / 4 * 4);
    float *sums = static_cast<float *>(workspace);
    uint16_t *counts = parts > 1 ? reinterpret_cast<uint16_t *>(sums + each) : nullptr;
    int32_t *tokens = parts > 1 ? reinterpret_cast<int32_t *>(counts + each) : nullptr;
    dispatch(E, logits_type, score, [&](auto n, auto s, auto element) {
        hipLaunchKernelGGL((balance_parts_kernel<decltype(n)::value, decltype(s)::value, decltype(element)>), dim3(parts),
                           dim3(kPartThreads), 0, stream, static_cast<const uint8_t *>(logits), logits_stride_bytes, topk_idx,
                           S, K, E, per, coef, loss, num_tokens_per_expert, num_tokens, sums, counts, tokens);
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || parts == 1) return e;
    int groups = 1;
    while (4 * groups < E) groups *= 2;
    hipLaunchKernelGGL(balance_finish_kernel, dim3(1), dim3(kFinishThreads), 0, stream, sums, counts, tokens, parts, E,
                       groups, coef, loss, num_tokens_per_expert, num_tokens);
    return hipGetLastError();
}

hipError_t launch_balance_loss_backward(const float *d_loss, const void *logits,
                                        int64_t logits_stride_bytes, int32_t logits_type,
                                        const int32_t *topk_idx,
                                        const int32_t *num_tokens_per_expert,
                                        const int32_t *num_tokens, int32_t S, int32_t K, int32_t E,
                                        int32_t score, float coef, void *d_logits,
                                        hipStream_t stream) {
    const int need = (S + kWaves - 1) / kWaves, grid = need < kBackwardGrid ? need : kBackwardGrid;
    dispatch(E, logits_type, score, [&](auto n, auto s, auto element) {
        using T = decltype(element);
        hipLaunchKernelGGL((balance_backward_kernel<decltype(n)::value, decltype(s)::value, T>), dim3(grid), dim3(kThreads),
                           0, stream, d_loss, static_cast<const uint8_t *>(logits), logits_stride_bytes, topk_idx,
                           num_tokens_per_expert, num_tokens, S, K, E, coef, static_cast<T *>(d_logits));
    });
    return hipGetLastError();
}

}  // namespace moe
