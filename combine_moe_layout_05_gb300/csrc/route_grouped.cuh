// route_grouped.cuh -- what the grouped router's kernel and its gradient share:
// the arguments and the scores.
#pragma once

#include "route_common.cuh"

namespace moe {
namespace {

// The logistic function of x and of -x: one power of 2 of -|x|, one reciprocal.
// Errors, with u = 2^-24: the product with log2(e) 1.22 |x| u and its power 4 u of
// the power, the sum u, the reciprocal 2 u, the product u: at most (1.22 |x| + 8) u
// of either value.  x = -inf: 0 and 1.
__device__ __forceinline__ float logistic(float x, float &rest)
{
    const float e = exp2_approx(-fabsf(x) * kLog2e), r = rcp_approx(1.0f + e), q = e * r;
    rest = x >= 0.0f ? q : r;
    return x >= 0.0f ? r : q;
}

}  // namespace
}  // namespace moe

// As MOE_ROUTE_CASES, with fewer widths: rows off the 16-byte grid value by value.
#define MOE_GROUPED_CASES(CALL, OTHER)                                          \
    if (bf16) {                                                                 \
        using L = __nv_bfloat16;                                                \
        if (rows_aligned(logits, OTHER, E, 2, 16)) {                            \
            if (E <= 256) return CALL(8, 8, L);                                 \
            if (E <= 512) return CALL(16, 8, L);                                \
            return CALL(32, 8, L);                                              \
        }                                                                       \
        if (E <= 256) return CALL(8, 1, L);                                     \
        return CALL(32, 1, L);                                                  \
    }                                                                           \
    if (rows_aligned(logits, OTHER, E, 4, 16)) {                                \
        if (E <= 128) return CALL(4, 4, float);                                 \
        if (E <= 256) return CALL(8, 4, float);                                 \
        if (E <= 384) return CALL(12, 4, float);                                \
        if (E <= 512) return CALL(16, 4, float);                                \
        return CALL(32, 4, float);                                              \
    }                                                                           \
    if (E <= 256) return CALL(8, 1, float);                                     \
    return CALL(32, 1, float)
