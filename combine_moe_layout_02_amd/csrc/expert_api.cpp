// C ABI of the calls around the experts (declared in include/moe.h): the gradients of the combine and the
// dispatch, MX rows, 8-bit checkpoints and the experts' product. As in moe_api.cpp, every check runs before
// the first HIP call, so a rejected call enqueues nothing.

#include <stdint.h>

#include "abi_checks.h"
#include "moe_internal.h"

namespace {

using namespace moe::checks;

// H of MX rows: blocks of 32 values, no partial block.
int check_mx_hidden(int32_t H) {
    const int st = check_hidden(H);
    if (st != MOE_OK) return st;
    return H % 32 == 0 ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

bool valid_format(int32_t format) { return format == MOE_MX_E2M1 || format == MOE_MX_E4M3; }

int64_t row_bytes(int32_t H, int32_t format) { return format == MOE_MX_E2M1 ? H / 2 : H; }

// A buffer's bytes [base, base + bytes), for the overlap checks. Rows at a stride end with the last row.
struct Span {
    const void *base;
    int64_t bytes;
};

Span rows_span(const void *base, int64_t rows, int64_t stride, int64_t row) {
    return Span{base, rows > 0 ? (rows - 1) * stride + row : 0};
}

bool overlap(const Span &a, const Span &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.base), y = reinterpret_cast<uintptr_t>(b.base);
    if (a.bytes <= 0 || b.bytes <= 0) return false;
    return x < y ? y - x < (uint64_t)a.bytes : x - y < (uint64_t)b.bytes;
}

// True when an output overlaps an input or another output.
template <int NI, int NO>
bool outputs_overlap(const Span (&in)[NI], const Span (&out)[NO]) {
    for (int i = 0; i < NO; ++i) {
        for (const Span &s : in)
            if (overlap(out[i], s)) return true;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return true;
    }
    return false;
}

// bf16 rows of H values at a stride.
int check_rows(const void *rows, int64_t stride, int64_t count, int32_t H) {
    if (count < 0 || stride < 2 * (int64_t)H || !extent_fits(count, stride)) return MOE_ERR_ARG;
    if (stride % 16 != 0 || !aligned(rows, 16)) return MOE_ERR_ALIGN;
    return MOE_OK;
}

int check_sizes(int32_t S, int32_t H, int32_t K, bool mx) {
    const int st = check_tokens(S, K);
    if (st != MOE_OK) return st;
    return mx ? check_mx_hidden(H) : check_hidden(H);
}

// What both combine gradients check besides the rows they read.
int check_gradient(const void *dy, int64_t expert_rows, const int32_t *slot_idx,
                   const float *topk_weights, int32_t H, const void *d_expert_out,
                   int64_t d_row_stride_bytes, const float *d_topk_weights) {
    const int st = check_rows(d_expert_out, d_row_stride_bytes, expert_rows, H);
    if (st != MOE_OK) return st;
    if (!aligned(dy, 16) || !aligned(slot_idx, 4) || !aligned(topk_weights, 4) ||
        !aligned(d_topk_weights, 4))
        return MOE_ERR_ALIGN;
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_combine_backward(const void *dy, const void *expert_out, int64_t row_stride_bytes,
                         int64_t expert_rows, const int32_t *slot_idx, const float *topk_weights,
                         int32_t S, int32_t H, int32_t K, void *d_expert_out,
                         int64_t d_row_stride_bytes, float *d_topk_weights, hipStream_t stream) {
    if (!dy || !expert_out || !slot_idx || !topk_weights || !d_expert_out || !d_topk_weights)
        return MOE_ERR_ARG;
    int st = check_sizes(S, H, K, false);
    if (st != MOE_OK) return st;
    st = check_rows(expert_out, row_stride_bytes, expert_rows, H);
    if (st != MOE_OK) return st;
    st = check_gradient(dy, expert_rows, slot_idx, topk_weights, H, d_expert_out,
                        d_row_stride_bytes, d_topk_weights);
    if (st != MOE_OK) return st;
    const int64_t table = (int64_t)S * K * 4;
    const Span in[] = {{dy, (int64_t)S * H * 2},
                       rows_span(expert_out, expert_rows, row_stride_bytes, 2 * (int64_t)H),
                       {slot_idx, table}, {topk_weights, table}};
    const Span out[] = {rows_span(d_expert_out, expert_rows, d_row_stride_bytes, 2 * (int64_t)H),
                        {d_topk_weights, table}};
    if (outputs_overlap(in, out)) return MOE_ERR_ARG;
    return from_hip(moe::launch_combine_backward(dy, expert_out, row_stride_bytes, expert_rows,
                                                 slot_idx, topk_weights, S, H, K, d_expert_out,
                                                 d_row_stride_bytes, d_topk_weights, stream));
}

int moe_combine_backward_mx(const void *dy, const void *codes, const void *scales,
                            int64_t expert_rows, const int32_t *slot_idx,
                            const float *topk_weights, int32_t S, int32_t H, int32_t K,
                            void *d_expert_out, int64_t d_row_stride_bytes,
                            float *d_topk_weights, hipStream_t stream) {
    if (!dy || !codes || !scales || !slot_idx || !topk_weights || !d_expert_out || !d_topk_weights)
        return MOE_ERR_ARG;
    int st = check_sizes(S, H, K, true);
    if (st != MOE_OK) return st;
    st = check_gradient(dy, expert_rows, slot_idx, topk_weights, H, d_expert_out,
                        d_row_stride_bytes, d_topk_weights);
    if (st != MOE_OK) return st;
    if (!aligned(codes, 16)) return MOE_ERR_ALIGN;
    const int64_t table = (int64_t)S * K * 4;
    const Span in[] = {{dy, (int64_t)S * H * 2}, {codes, expert_rows * H},
                       {scales, expert_rows * (H / 32)}, {slot_idx, table}, {topk_weights, table}};
    const Span out[] = {rows_span(d_expert_out, expert_rows, d_row_stride_bytes, 2 * (int64_t)H),
                        {d_topk_weights, table}};
    if (outputs_overlap(in, out)) return MOE_ERR_ARG;
    return from_hip(moe::launch_combine_backward_mx(dy, codes, scales, expert_rows, slot_idx,
                                                    topk_weights, S, H, K, d_expert_out,
                                                    d_row_stride_bytes, d_topk_weights, stream));
}

int moe_dispatch_backward(const void *d_rows, int64_t row_stride_bytes, int64_t expert_rows,
                          const int32_t *slot_idx, int32_t S, int32_t H, int32_t K, void *dx,
                          hipStream_t stream) {
    if (!d_rows || !slot_idx || !dx) return MOE_ERR_ARG;
    int st = check_sizes(S, H, K, false);
    if (st != MOE_OK) return st;
    st = check_rows(d_rows, row_stride_bytes, expert_rows, H);
    if (st != MOE_OK) return st;
    if (!aligned(slot_idx, 4) || !aligned(dx, 16)) return MOE_ERR_ALIGN;
    const Span in[] = {rows_span(d_rows, expert_rows, row_stride_bytes, 2 * (int64_t)H),
                       {slot_idx, (int64_t)S * K * 4}};
    const Span out[] = {{dx, (int64_t)S * H * 2}};
    if (outputs_overlap(in, out)) return MOE_ERR_ARG;
    return from_hip(moe::launch_dispatch_backward(d_rows, row_stride_bytes, expert_rows, slot_idx,
                                                  S, H, K, dx, stream));
}

int moe_combine_checkpoint(const void *expert_out, int64_t row_stride_bytes, int64_t expert_rows,
                           const int32_t *slot_idx, const float *topk_weights, int32_t S,
                           int32_t H, int32_t K, void *y, void *codes, void *scales,
                           hipStream_t stream) {
    if (!expert_out || !slot_idx || !topk_weights || !y || !codes || !scales) return MOE_ERR_ARG;
    int st = check_sizes(S, H, K, true);
    if (st != MOE_OK) return st;
    st = check_rows(expert_out, row_stride_bytes, expert_rows, H);
    if (st != MOE_OK) return st;
    if (!aligned(slot_idx, 4) || !aligned(topk_weights, 4) || !aligned(y, 16) || !aligned(codes, 16))
        return MOE_ERR_ALIGN;
    const int64_t table = (int64_t)S * K * 4;
    const Span in[] = {rows_span(expert_out, expert_rows, row_stride_bytes, 2 * (int64_t)H),
                       {slot_idx, table}, {topk_weights, table}};
    const Span out[] = {{y, (int64_t)S * H * 2}, {codes, expert_rows * H},
                        {scales, expert_rows * (H / 32)}};
    if (outputs_overlap(in, out)) return MOE_ERR_ARG;
    return from_hip(moe::launch_combine_checkpoint(expert_out, row_stride_bytes, expert_rows,
                                                   slot_idx, topk_weights, S, H, K, y, codes,
                                                   scales, stream));
}

int64_t moe_mx_row_bytes(int32_t H, int32_t format) {
    const int st = check_mx_hidden(H);
    if (st != MOE_OK) return st;
    if (!valid_format(format)) return MOE_ERR_ARG;
    return row_bytes(H, format);
}

int moe_mx_quantize(const void *rows, int64_t row_stride_bytes, const int32_t *num_rows,
                    int64_t max_rows, int32_t H, int32_t format, void *codes, void *scales,
                    hipStream_t stream) {
    if (!rows || !codes || !scales) return MOE_ERR_ARG;
    int st = check_mx_hidden(H);
    if (st != MOE_OK) return st;
    if (!valid_format(format) || max_rows > MOE_MAX_OUT_ROWS) return MOE_ERR_ARG;
    st = check_rows(rows, row_stride_bytes, max_rows, H);
    if (st != MOE_OK) return st;
    if (!aligned(num_rows, 4) || !aligned(codes, 16)) return MOE_ERR_ALIGN;
    const Span in[] = {rows_span(rows, max_rows, row_stride_bytes, 2 * (int64_t)H),
                       {num_rows, num_rows ? 4 : 0}};
    const Span out[] = {{codes, max_rows * row_bytes(H, format)}, {scales, max_rows * (H / 32)}};
    if (outputs_overlap(in, out)) return MOE_ERR_ARG;
    return from_hip(moe::launch_mx_quantize(rows, row_stride_bytes, num_rows, max_rows, H, format,
                                            codes, scales, stream));
}

int moe_mx_dequantize(const void *codes, const void *scales, const int32_t *num_rows,
                      int64_t max_rows, int32_t H, int32_t format, void *rows,
                      int64_t row_stride_bytes, hipStream_t stream) {
    if (!rows || !codes || !scales) return MOE_ERR_ARG;
    int st = check_mx_hidden(H);
    if (st != MOE_OK) return st;
    if (!valid_format(format) || max_rows > MOE_MAX_OUT_ROWS) return MOE_ERR_ARG;
    st = check_rows(rows, row_stride_bytes, max_rows, H);
    if (st != MOE_OK) return st;
    if (!aligned(num_rows, 4) || !aligned(codes, 16)) return MOE_ERR_ALIGN;
    const Span in[] = {{codes, max_rows * row_bytes(H, format)}, {scales, max_rows * (H / 32)},
                       {num_rows, num_rows ? 4 : 0}};
    const Span out[] = {rows_span(rows, max_rows, row_stride_bytes, 2 * (int64_t)H)};
    if (outputs_overlap(in, out)) return MOE_ERR_ARG;
    return from_hip(moe::launch_mx_dequantize(codes, scales, num_rows, max_rows, H, format, rows,
                                              row_stride_bytes, stream));
}

int moe_mx_product(const void *a_codes, const void *a_scales, int64_t a_rows,
                   const int32_t *group_base, int32_t G, const void *w_codes, const void *w_scales,
                   int32_t O, int32_t H, int32_t epilogue, void *out, int64_t out_stride_bytes,
                   hipStream_t stream) {
    if (!a_codes || !a_scales || !group_base || !w_codes || !w_scales || !out) return MOE_ERR_ARG;
    int st = check_mx_hidden(H);
    if (st != MOE_OK) return st;
    if (a_rows < 0 || a_rows > MOE_MAX_OUT_ROWS || G < 1 || G > MOE_MAX_EXPERTS || O < 1 ||
        O > MOE_MAX_OUTPUTS)
        return MOE_ERR_ARG;
    if (epilogue != MOE_MX_PLAIN && epilogue != MOE_MX_GATED) return MOE_ERR_ARG;
    if (epilogue == MOE_MX_GATED && O % 2 != 0) return MOE_ERR_UNSUPPORTED;
    const int64_t out_bytes = 2 * (int64_t)(epilogue == MOE_MX_GATED ? O / 2 : O);
    if (out_stride_bytes < out_bytes || !extent_fits(a_rows, out_stride_bytes)) return MOE_ERR_ARG;
    if (out_stride_bytes % 2 != 0 || !aligned(out, 2) || !aligned(a_codes, 16) ||
        !aligned(w_codes, 16) || !aligned(group_base, 4))
        return MOE_ERR_ALIGN;
    const int64_t w_rows = (int64_t)G * O;
    const Span in[] = {{a_codes, a_rows * (H / 2)}, {a_scales, a_rows * (H / 32)},
                       {group_base, 4 * ((int64_t)G + 1)}, {w_codes, w_rows * (H / 2)},
                       {w_scales, w_rows * (H / 32)}};
    const Span outs[] = {rows_span(out, a_rows, out_stride_bytes, out_bytes)};
    if (outputs_overlap(in, outs)) return MOE_ERR_ARG;
    return from_hip(moe::launch_mx_product(a_codes, a_scales, a_rows, group_base, G, w_codes,
                                           w_scales, O, H, epilogue, out, out_stride_bytes, stream));
}

}  // extern "C"
