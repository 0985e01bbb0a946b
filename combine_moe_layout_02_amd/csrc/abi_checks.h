// Argument checks shared by the C ABI layers (moe_api.cpp, expert_api.cpp, layer_api.cpp). Host only, no HIP call.
#pragma once

#include "moe_internal.h"

namespace moe {
namespace checks {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int check_hidden(int32_t H) {
    if (H < 16 || H > MOE_MAX_HIDDEN) return MOE_ERR_ARG;
    if (H % 16 != 0) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

inline int check_tokens(int32_t S, int32_t K) {
    if (S < 1 || K < 1 || K > MOE_MAX_K) return MOE_ERR_ARG;
    if (S > MOE_MAX_TOKENS) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

inline int from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// True when rows [0, rows) at `stride` bytes apart have byte offsets an int64 can hold (rows * stride
// <= INT64_MAX), so the kernels' row addresses cannot wrap.
inline bool extent_fits(int64_t rows, int64_t stride) {
    return rows <= 1 || stride <= INT64_MAX / rows;
}

// A buffer's bytes [base, base + bytes), for the overlap checks. Rows at a stride end with the last row.
struct Span {
    const void *base;
    int64_t bytes;
};

inline Span rows_span(const void *base, int64_t rows, int64_t stride, int64_t row) {
    return Span{base, rows > 0 ? (rows - 1) * stride + row : 0};
}

inline bool overlap(const Span &a, const Span &b) {
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
inline int check_rows(const void *rows, int64_t stride, int64_t count, int32_t H) {
    if (count < 0 || stride < 2 * (int64_t)H || !extent_fits(count, stride)) return MOE_ERR_ARG;
    if (stride % 16 != 0 || !aligned(rows, 16)) return MOE_ERR_ALIGN;
    return MOE_OK;
}

}  // namespace checks
}  // namespace moe
