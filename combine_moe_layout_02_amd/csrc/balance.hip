// The router's balance loss over the experts' counts, and its gradient, for gfx950 (see moe_balance_loss in moe.h).
//
// A wave takes a token: lane l holds experts l, l + 64, ... of it, so that its scores are two reductions over the wave's
// lanes, and their sums over tokens stay in its registers. The exponentials and the reductions' chains bound it, and launches.
// Calls one after another in a graph, us with a softmax and with sigmoids: 8192 tokens of 256 experts (8.4 MB) 9.9 and 10.2 forward
// (5.8 in the parts, 5.0 in the joining kernel) and 5.9 and 6.2 back, 65536 of them 20.6 and 23.1, 24.9 and 26.0, 128 tokens of 16
// experts (one part) 5.8 and 6.6, 2.3 and 2.3. 8192 tokens in parts of 64 take 10.6 and 11.2, of 128 13.5 and 14.7. With the library's
// expf 65536 tokens take 22.7 and 30.7, 25.3 and 30.6; with loads and stores that a test keeps in the row, not the buffer's
// end, 2.8 more. The gradient with 1024 workgroups takes 5.7 and 6.2 (65536 tokens 25.4 and 28.4), with 512 5.9 and 6.7 (29.5 and 34.5),
// with 4096 the same.

#include "pack_rows.h"
#include "wave_ops.h"

namespace moe {
namespace {

typedef __bf16 bf16_t;

constexpr int kPartThreads = 1024, kPartWaves = kPartThreads / 64;
constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kFinishThreads = 1024;
constexpr int kBackwardGrid = 2048;

// exp(x) to 2 ulp for x in [-87.3, 0], from the hardware's exp2 of x * log2(e) and the rest of that product; 0 below, where exp(x)
// is less than 2^-126 and the hardware gives no subnormals; NaN of a NaN. -200 keeps the rest of -inf a number. A third of
// the library function's instructions, which bound these kernels. What is taken as 0 is a score that far below the largest, or 1 -
// sigmoid(l) of l > 87.3.
__device__ inline float exp_of(float x) {
    constexpr float kLog2e = 1.44269502e+00f, kLog2eRest = 1.92596299e-08f, kLn2 = 6.93147182e-01f;
    x = x < -200.0f ? -200.0f : x;
    const float t = x * kLog2e;
    const float rest = __builtin_fmaf(x, kLog2eRest, __builtin_fmaf(x, kLog2e, -t));
    const float y = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(y, rest * kLn2, y);
}

// The scores of one token from its logits (-inf past E): exp(l - max) over their sum, or sigmoids over theirs. Where all
// logits are below zero the sigmoids, exp(l) / (1 + exp(l)), are taken against exp(max): a token far below zero keeps its scores,
// also those far below its largest. A logit of -inf has score 0, also where there is no other. turn: 1 - sigmoid(l), for
// MOE_SCORE_SIGMOID.
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
            s[i] = (top < 0.0f ? exp_of(l[i] - top) : l[i] > 0.0f ? 1.0f : far) * share;
        } else {
            s[i] = exp_of(l[i] - top);
        }
        sum += s[i];
    }
    const float each = 1.0f / wave::sum(sum);
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = l[i] == -__builtin_inff() ? 0.0f : s[i] * each;
}

// A token's logits (-inf past E) and entries (-1 past K) in a wave's lanes; nothing of tokens past the end. Lanes past a row's
// end read nothing: the buffer ends there.
template <int N, class T>
struct Token {
    float l[N];
    int id;
    __device__ void load(const uint8_t *__restrict__ logits, int64_t stride, const int32_t *__restrict__ topk, int t, int end, int K, int E) {
        const int lane = threadIdx.x & 63, bytes = t < end ? E * (int)sizeof(T) : 0;
        const __amdgpu_buffer_rsrc_t row = rows::rsrc(logits + t * stride, bytes);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (lane + 64 * i) * (int)sizeof(T);
            float v;
            if constexpr (sizeof(T) == 4) v = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(row, at, 0, 0));
            else v = __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b16(row, at, 0, 0) << 16);
            l[i] = at < bytes ? v : -__builtin_inff();
        }
        const int entries = t < end ? K : 0;
        const int e = __builtin_amdgcn_raw_buffer_load_b32(rows::rsrc(topk + (int64_t)t * K, entries * 4), lane * 4, 0, 0);
        id = lane < entries ? e : -1;
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
    float *__restrict__ part_sums, uint16_t *__restrict__ part_counts, int32_t *__restrict__ part_tokens,
    BalanceShares *__restrict__ shares) {
    __shared__ int32_t count[64 * N];
    __shared__ float sums[kPartWaves][64 * N];
    __shared__ int32_t live[kPartWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
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
        if (tid == 0 && blockIdx.x == 0) shares->done = 0;  // for the joining kernel
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

// Workgroup w joins the parts' sums and counts of experts [64 w, 64 w + 64): 16 lanes four experts each of every 64th part, four
// such rows a wave, then the waves' in order. Each leaves its share of the loss, and the last to come adds the shares in
// their order, whichever it is. (One workgroup for all experts read 393 KB, of 256 parts of 256 experts, at 33 bytes a cycle: 7 us.)
__global__ __launch_bounds__(kFinishThreads) void balance_finish_kernel(
    const float *__restrict__ part_sums, const uint16_t *__restrict__ part_counts,
    const int32_t *__restrict__ part_tokens, int parts, int E, float coef, BalanceShares *__restrict__ shares,
    float *__restrict__ loss, int32_t *__restrict__ counts, int32_t *__restrict__ tokens) {
    constexpr int kFinishWaves = kFinishThreads / 64;
    __shared__ __align__(16) float sums[kFinishWaves][64];
    __shared__ __align__(16) int32_t count[kFinishWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wide = (E + 3) / 4 * 4, e0 = blockIdx.x * 64, mine = (lane & 15) * 4, e = e0 + mine;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int c[4] = {0, 0, 0, 0}, live = 0;
    // parts past the last read as zero, where the buffers end
    const __amdgpu_buffer_rsrc_t sum_src = rows::rsrc(part_sums, parts * wide * 4), count_src = rows::rsrc(part_counts, parts * wide * 2);
#pragma unroll
    for (int k = 0; k < kBalanceParts / (4 * kFinishWaves); ++k) {
        const int p = wave * 4 + (lane >> 4) + k * 4 * kFinishWaves, at = e < wide ? p * wide + e : 1 << 28;
        const rows::u32x4 f = rows::load16(sum_src, at * 4);
        const auto n = __builtin_amdgcn_raw_buffer_load_b64(count_src, at * 2, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[i] += __uint_as_float(f[i]);
            c[i] += (int)(n[i >> 1] >> (16 * (i & 1)) & 0xFFFFu);
        }
    }
    if (wave == 0)
        for (int p = lane; p < parts; p += 64) live += part_tokens[p];
    const auto add = [](auto a, auto b) { return a + b; };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s[i] = wave::join<false>(wave::join<true>(s[i], add), add);
        c[i] = wave::join<false>(wave::join<true>(c[i], add), add);
    }
    if (lane < 16) {
        *reinterpret_cast<float4 *>(&sums[wave][mine]) = float4{s[0], s[1], s[2], s[3]};
        *reinterpret_cast<int4 *>(&count[wave][mine]) = int4{c[0], c[1], c[2], c[3]};
    }
    __syncthreads();
    if (wave > 0) return;
    float sum = 0.0f;
    int all = 0;
#pragma unroll
    for (int w = 0; w < kFinishWaves; ++w) sum += sums[w][lane], all += count[w][lane];
    if (e0 + lane < E) counts[e0 + lane] = all;
    double part = wave::sum((double)all * (double)sum);
    all = wave::sum(all);
    live = wave::sum(live);
    if (lane > 0) return;
    if (gridDim.x > 1) {
        __hip_atomic_store(&shares->share[blockIdx.x], part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(&shares->entries[blockIdx.x], all, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const int before = __hip_atomic_fetch_add(&shares->done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
        if (before != (int)gridDim.x - 1) return;
        part = 0.0;
        all = 0;
        for (int w = 0; w < (int)gridDim.x; ++w) {
            part += __hip_atomic_load(&shares->share[w], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            all += __hip_atomic_load(&shares->entries[w], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    *loss = loss_of(part, all, live, E, coef);
    *tokens = live;
}

// A wave a token, as above. n[e] counts from the mean, which takes nothing from the gradient (the scores' sum is 1), and
// lets equal counts cancel exactly.
template <int N, int SCORE, class T>
__global__ __launch_bounds__(kThreads) void balance_backward_kernel(
    const float *__restrict__ d_loss, const uint8_t *__restrict__ logits, int64_t stride,
    const int32_t *__restrict__ topk, const int32_t *__restrict__ counts, const int32_t *__restrict__ tokens, int S,
    int K, int E, float coef, T *__restrict__ d_logits) {
    const int lane = threadIdx.x & 63, step = gridDim.x * kWaves;
    int n[N];
    double sum = 0.0;  // counts of many GPUs may pass 32 bits together
#pragma unroll
    for (int i = 0; i < N; ++i) {
        n[i] = lane + 64 * i < E ? counts[lane + 64 * i] : 0;
        sum += n[i];
    }
    sum = wave::sum(sum);
    const int mean = (int)(sum / E);
    const double all = sum * (double)*tokens;
    // coef, d_loss and 1 / (N T) may each be near an end of fp32's range: the factor is taken in 64 bits, its mantissa meets the
    // counts and its exponent the result
    int power;
    const double each = __builtin_frexp(all > 0.0 ? (double)coef * E / all * *d_loss : 0.0, &power);
    float g[N];
#pragma unroll
    for (int i = 0; i < N; ++i) g[i] = (float)(each * (n[i] - mean));
    int t = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Token<N, T> next;
    next.load(logits, stride, topk, t, S, K, E);
    for (; t < S; t += step) {
        const Token<N, T> token = next;
        next.load(logits, stride, topk, t + step, S, K, E);
        const bool lives = __any(token.id >= 0 && token.id < E);
        float s[N], turn[N];
        scores_of<N, SCORE>(token.l, s, turn);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) dot += g[i] * s[i];
        dot = wave::sum(dot);
        const __amdgpu_buffer_rsrc_t dst = rows::rsrc(d_logits + (int64_t)t * E, E * (int)sizeof(T));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float d = s[i] * (g[i] - dot);
            if (SCORE == MOE_SCORE_SIGMOID) d *= turn[i];
            d = lives ? __builtin_ldexpf(d, power) : 0.0f;
            const int at = (lane + 64 * i) * (int)sizeof(T);
            if constexpr (sizeof(T) == 4) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(d), dst, at, 0, 0);
            else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (T)d), dst, at, 0, 0);
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
    const int most = balance_parts(S, E), per = (S + most - 1) / most, parts = (S + per - 1) / per;
    const int64_t each = (int64_t)most * ((E + 3) / 4 * 4);
    BalanceShares *const shares = static_cast<BalanceShares *>(workspace);
    float *const sums = parts > 1 ? reinterpret_cast<float *>(shares + 1) : nullptr;
    uint16_t *const counts = parts > 1 ? reinterpret_cast<uint16_t *>(sums + each) : nullptr;
    int32_t *const tokens = parts > 1 ? reinterpret_cast<int32_t *>(counts + each) : nullptr;
    dispatch(E, logits_type, score, [&](auto n, auto s, auto element) {
        hipLaunchKernelGGL((balance_parts_kernel<decltype(n)::value, decltype(s)::value, decltype(element)>), dim3(parts),
                           dim3(kPartThreads), 0, stream, static_cast<const uint8_t *>(logits), logits_stride_bytes, topk_idx,
                           S, K, E, per, coef, loss, num_tokens_per_expert, num_tokens, sums, counts, tokens, shares);
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || parts == 1) return e;
    hipLaunchKernelGGL(balance_finish_kernel, dim3((E + 63) / 64), dim3(kFinishThreads), 0, stream, sums, counts, tokens,
                       parts, E, coef, shares, loss, num_tokens_per_expert, num_tokens);
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
