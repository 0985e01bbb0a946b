// C ABI of the 8-bit layer around the dispatch (declared in include/moe.h): rows in 8 bits, the experts' INT8
// product, the RMS norm and the balance loss, with their gradients. As in moe_api.cpp, every check runs before
// the first HIP call, so a rejected call enqueues nothing.

#include <cmath>
#include <stdint.h>

#include "abi_checks.h"
#include "moe_internal.h"

namespace {

using namespace moe::checks;

bool valid_float(int32_t type) { return type == MOE_BF16 || type == MOE_FP32; }
int64_t float_bytes(int32_t type) { return type == MOE_BF16 ? 2 : 4; }
bool in_8_bits(int32_t quant) { return moe::valid_quant(quant) && quant != MOE_QUANT_NONE; }

// rows of a call whose row buffers may be NULL where it has none
int check_count(int64_t rows) { return rows < 0 || rows > MOE_MAX_OUT_ROWS ? MOE_ERR_ARG : MOE_OK; }

// What both conversions check; the bf16 side and the 8-bit side of the same rows.
int check_row8(const void *rows, int64_t stride, const int32_t *num_rows, int64_t max_rows,
               int32_t H, int32_t quant, const void *codes, const float *scales) {
    int st = check_hidden(H);
    if (st != MOE_OK) return st;
    if (!in_8_bits(quant)) return MOE_ERR_ARG;
    st = check_count(max_rows);
    if (st != MOE_OK) return st;
    if (max_rows > 0 && (!rows || !codes || !scales)) return MOE_ERR_ARG;
    st = check_rows(rows, stride, max_rows, H);
    if (st != MOE_OK) return st;
    if (!aligned(num_rows, 4) || !aligned(codes, 16) || !aligned(scales, 4)) return MOE_ERR_ALIGN;
    return MOE_OK;
}

// S, K, E, the logits' type and rows, and the score.
int check_router(const void *logits, int64_t stride, int32_t type, const int32_t *topk_idx, int32_t S,
                 int32_t K, int32_t E, int32_t score, float coef) {
    if (!logits || !topk_idx) return MOE_ERR_ARG;
    const int st = check_tokens(S, K);
    if (st != MOE_OK) return st;
    if (E < 1 || E > MOE_MAX_EXPERTS || !valid_float(type) || !std::isfinite(coef)) return MOE_ERR_ARG;
    if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_ERR_ARG;
    const int64_t size = float_bytes(type);
    if (stride < size * E || !extent_fits(S, stride)) return MOE_ERR_ARG;
    if (stride % size != 0 || !aligned(logits, (uintptr_t)size) || !aligned(topk_idx, 4))
        return MOE_ERR_ALIGN;
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_row_quantize(const void *rows, int64_t row_stride_bytes, const int32_t *num_rows,
                     int64_t max_rows, int32_t H, int32_t quant, void *codes, float *scales,
                     hipStream_t stream) {
    const int st = check_row8(rows, row_stride_bytes, num_rows, max_rows, H, quant, codes, scales);
    if (st != MOE_OK) return st;
    const Span in[] = {rows_span(rows, max_rows, row_stride_bytes, 2 * (int64_t)H),
                       {num_rows, num_rows ? 4 : 0}};
    const Span out[] = {{codes, max_rows * H}, {scales, max_rows * 4}};
    if (outputs_overlap(in, out)) return MOE_ERR_ARG;
    return from_hip(moe::launch_row_quantize(rows, row_stride_bytes, num_rows, max_rows, H, quant,
                                             codes, scales, stream));
}

int moe_row_dequantize(const void *codes, const float *scales, const int32_t *num_rows,
                       int64_t max_rows, int32_t H, int32_t quant, void *rows,
                       int64_t row_stride_bytes, hipStream_t stream) {
    const int st = check_row8(rows, row_stride_bytes, num_rows, max_rows, H, quant, codes, scales);
    if (st != MOE_OK) return st;
    const Span in[] = {{codes, max_rows * H}, {scales, max_rows * 4}, {num_rows, num_rows ? 4 : 0}};
    const Span out[] = {rows_span(rows, max_rows, row_stride_bytes, 2 * (int64_t)H)};
    if (outputs_overlap(in, out)) return MOE_ERR_ARG;
    return from_hip(moe::launch_row_dequantize(codes, scales, num_rows, max_rows, H, quant, rows,
                                               row_stride_bytes, stream));
}

int moe_scaled_product(const void *a_codes, const float *a_scales, int64_t a_rows,
                       const int32_t *group_base, int32_t G, const void *w_codes,
                       const float *w_scales, int32_t O, int32_t H, int32_t epilogue, void *out,
                       int64_t out_stride_bytes, hipStream_t stream) {
    int st = check_hidden(H);
    if (st != MOE_OK) return st;
    st = check_count(a_rows);
    if (st != MOE_OK) return st;
    if (!group_base || !w_codes || !w_scales) return MOE_ERR_ARG;
    if (a_rows > 0 && (!a_codes || !a_scales || !out)) return MOE_ERR_ARG;
    if (G < 1 || G > MOE_MAX_EXPERTS || O < 1 || O > MOE_MAX_OUTPUTS) return MOE_ERR_ARG;
    if (epilogue != MOE_MX_PLAIN && epilogue != MOE_MX_GATED) return MOE_ERR_ARG;
    if (epilogue == MOE_MX_GATED && O % 2 != 0) return MOE_ERR_UNSUPPORTED;
    const int64_t out_bytes = 2 * (int64_t)(epilogue == MOE_MX_GATED ? O / 2 : O);
    if (out_stride_bytes < out_bytes || !extent_fits(a_rows, out_stride_bytes)) return MOE_ERR_ARG;
    if (out_stride_bytes % 2 != 0 || !aligned(out, 2) || !aligned(a_codes, 16) ||
        !aligned(a_scales, 4) || !aligned(w_codes, 16) || !aligned(w_scales, 4) ||
        !aligned(group_base, 4))
        return MOE_ERR_ALIGN;
    const int64_t w_rows = (int64_t)G * O;
    const Span in[] = {{a_codes, a_rows * H}, {a_scales, a_rows * 4}, {group_base, 4 * ((int64_t)G + 1)},
                       {w_codes, w_rows * H}, {w_scales, w_rows * 4}};
    const Span outs[] = {rows_span(out, a_rows, out_stride_bytes, out_bytes)};
    if (outputs_overlap(in, outs)) return MOE_ERR_ARG;
    return from_hip(moe::launch_int8_product(a_codes, a_scales, a_rows, group_base, G, w_codes,
                                             w_scales, O, H, epilogue, out, out_stride_bytes, stream));
}

int moe_rms_norm(const void *x, int64_t x_stride_bytes, const void *residual,
                 int64_t residual_stride_bytes, const void *weight, int32_t weight_type, float eps,
                 int64_t rows, int32_t H, int32_t quant, void *sum, int64_t sum_stride_bytes,
                 void *out, void *codes, float *scales, hipStream_t stream) {
    int st = check_hidden(H);
    if (st != MOE_OK) return st;
    st = check_count(rows);
    if (st != MOE_OK) return st;
    if (!weight || !valid_float(weight_type) || !moe::valid_quant(quant)) return MOE_ERR_ARG;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return MOE_ERR_ARG;
    const bool quantised = quant != MOE_QUANT_NONE;
    if (!quantised && (codes || scales)) return MOE_ERR_ARG;
    if (rows > 0) {
        if (!x || (sum != nullptr) != (residual != nullptr)) return MOE_ERR_ARG;
        if (quantised ? !codes || !scales : !out) return MOE_ERR_ARG;
    }
    const int64_t row = 2 * (int64_t)H;
    st = check_rows(x, x_stride_bytes, rows, H);
    if (st == MOE_OK && residual) st = check_rows(residual, residual_stride_bytes, rows, H);
    if (st == MOE_OK && sum) st = check_rows(sum, sum_stride_bytes, rows, H);
    if (st != MOE_OK) return st;
    if (!aligned(weight, 16) || !aligned(out, 16) || !aligned(codes, 16) || !aligned(scales, 4))
        return MOE_ERR_ALIGN;
    // the sum may take the place of the rows that it is read from
    const bool over_x = sum == x && sum_stride_bytes == x_stride_bytes;
    const bool over_residual = sum == residual && sum_stride_bytes == residual_stride_bytes;
    const Span xs = rows_span(x, rows, x_stride_bytes, row);
    const Span rs = rows_span(residual, residual ? rows : 0, residual_stride_bytes, row);
    const Span ws = {weight, H * float_bytes(weight_type)};
    const Span sums = rows_span(sum, sum ? rows : 0, sum_stride_bytes, row);
    if ((!over_x && overlap(sums, xs)) || (!over_residual && overlap(sums, rs)) || overlap(sums, ws))
        return MOE_ERR_ARG;
    const Span in[] = {xs, rs, ws, sums};
    const Span outs[] = {{out, out ? rows * row : 0}, {codes, codes ? rows * H : 0},
                         {scales, scales ? rows * 4 : 0}};
    if (outputs_overlap(in, outs)) return MOE_ERR_ARG;
    return from_hip(moe::launch_rms_norm(x, x_stride_bytes, residual, residual_stride_bytes, weight,
                                         weight_type, eps, rows, H, quant, sum, sum_stride_bytes, out,
                                         codes, scales, stream));
}

int64_t moe_rms_norm_backward_workspace_bytes(int64_t rows, int32_t H) {
    int st = check_hidden(H);
    if (st == MOE_OK) st = check_count(rows);
    if (st != MOE_OK) return st;
    return moe::norm_workspace(rows, H);
}

int moe_rms_norm_backward(const void *dy, int64_t dy_stride_bytes, const void *sum,
                          int64_t sum_stride_bytes, const void *weight, int32_t weight_type,
                          float eps, const void *d_sum, int64_t d_sum_stride_bytes, int64_t rows,
                          int32_t H, void *dx, float *d_weight, void *workspace,
                          int64_t workspace_bytes, hipStream_t stream) {
    int st = check_hidden(H);
    if (st != MOE_OK) return st;
    st = check_count(rows);
    if (st != MOE_OK) return st;
    if (!weight || !valid_float(weight_type) || !d_weight) return MOE_ERR_ARG;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return MOE_ERR_ARG;
    if (rows > 0 && (!dy || !sum || !dx)) return MOE_ERR_ARG;
    const int64_t row = 2 * (int64_t)H;
    st = check_rows(dy, dy_stride_bytes, rows, H);
    if (st == MOE_OK) st = check_rows(sum, sum_stride_bytes, rows, H);
    if (st == MOE_OK && d_sum) st = check_rows(d_sum, d_sum_stride_bytes, rows, H);
    if (st != MOE_OK) return st;
    if (!aligned(weight, 16) || !aligned(dx, 16) || !aligned(d_weight, 16) || !aligned(workspace, 16))
        return MOE_ERR_ALIGN;
    const int64_t need = moe::norm_workspace(rows, H);
    if (workspace_bytes < need) return MOE_ERR_WINDOW;
    if (need > 0 && !workspace) return MOE_ERR_ARG;
    const Span in[] = {rows_span(dy, rows, dy_stride_bytes, row), rows_span(sum, rows, sum_stride_bytes, row),
                       {weight, H * float_bytes(weight_type)},
                       rows_span(d_sum, d_sum ? rows : 0, d_sum_stride_bytes, row)};
    const Span outs[] = {{dx, rows * row}, {d_weight, 4 * (int64_t)H}, {workspace, need}};
    if (outputs_overlap(in, outs)) return MOE_ERR_ARG;
    return from_hip(moe::launch_rms_norm_backward(dy, dy_stride_bytes, sum, sum_stride_bytes, weight,
                                                  weight_type, eps, d_sum, d_sum_stride_bytes, rows, H,
                                                  dx, d_weight, workspace, stream));
}

int64_t moe_balance_loss_workspace_bytes(int32_t S, int32_t E) {
    const int st = check_tokens(S, 1);
    if (st != MOE_OK) return st;
    if (E < 1 || E > MOE_MAX_EXPERTS) return MOE_ERR_ARG;
    return moe::balance_workspace(S, E);
}

int moe_balance_loss(const void *logits, int64_t logits_stride_bytes, int32_t logits_type,
                     const int32_t *topk_idx, int32_t S, int32_t K, int32_t E, int32_t score,
                     float coef, float *loss, int32_t *num_tokens_per_expert, int32_t *num_tokens,
                     void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (!loss || !num_tokens_per_expert || !num_tokens) return MOE_ERR_ARG;
    const int st = check_router(logits, logits_stride_bytes, logits_type, topk_idx, S, K, E, score, coef);
    if (st != MOE_OK) return st;
    if (!aligned(loss, 4) || !aligned(num_tokens_per_expert, 4) || !aligned(num_tokens, 4) ||
        !aligned(workspace, 16))
        return MOE_ERR_ALIGN;
    const int64_t need = moe::balance_workspace(S, E);
    if (workspace_bytes < need) return MOE_ERR_WINDOW;
    if (need > 0 && !workspace) return MOE_ERR_ARG;
    const Span in[] = {rows_span(logits, S, logits_stride_bytes, E * float_bytes(logits_type)),
                       {topk_idx, (int64_t)S * K * 4}};
    const Span outs[] = {{loss, 4}, {num_tokens_per_expert, 4 * (int64_t)E}, {num_tokens, 4},
                         {workspace, need}};
    if (outputs_overlap(in, outs)) return MOE_ERR_ARG;
    return from_hip(moe::launch_balance_loss(logits, logits_stride_bytes, logits_type, topk_idx, S, K, E,
                                             score, coef, loss, num_tokens_per_expert, num_tokens,
                                             workspace, stream));
}

int moe_balance_loss_backward(const float *d_loss, const void *logits, int64_t logits_stride_bytes,
                              int32_t logits_type, const int32_t *topk_idx,
                              const int32_t *num_tokens_per_expert, const int32_t *num_tokens,
                              int32_t S, int32_t K, int32_t E, int32_t score, float coef,
                              void *d_logits, hipStream_t stream) {
    if (!d_loss || !num_tokens_per_expert || !num_tokens || !d_logits) return MOE_ERR_ARG;
    const int st = check_router(logits, logits_stride_bytes, logits_type, topk_idx, S, K, E, score, coef);
    if (st != MOE_OK) return st;
    const int64_t size = float_bytes(logits_type);
    if (!aligned(d_loss, 4) || !aligned(num_tokens_per_expert, 4) || !aligned(num_tokens, 4) ||
        !aligned(d_logits, (uintptr_t)size))
        return MOE_ERR_ALIGN;
    const Span in[] = {{d_loss, 4}, rows_span(logits, S, logits_stride_bytes, E * size),
                       {topk_idx, (int64_t)S * K * 4}, {num_tokens_per_expert, 4 * (int64_t)E},
                       {num_tokens, 4}};
    const Span outs[] = {{d_logits, S * E * size}};
    if (outputs_overlap(in, outs)) return MOE_ERR_ARG;
    return from_hip(moe::launch_balance_loss_backward(d_loss, logits, logits_stride_bytes, logits_type,
                                                      topk_idx, num_tokens_per_expert, num_tokens, S, K,
                                                      E, score, coef, d_logits, stream));
}

}  // extern "C"
