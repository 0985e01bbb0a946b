// Argument checks shared by the C ABI layers (moe_api.cpp, expert_api.cpp). Host only, no HIP call.
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

}  // namespace checks
}  // namespace moe
