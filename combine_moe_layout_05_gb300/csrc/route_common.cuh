// route_common.cuh -- what the router's kernel and its gradient share: a row of
// logits in a warp's registers, the softmax's pieces, and the choice of a
// kernel's width by the row's length and alignment.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "moe_layout.h"

namespace moe {
namespace {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float from_float(float v, float) { return v; }
__device__ __forceinline__ __nv_bfloat16 from_float(float v, __nv_bfloat16) { return __float2bfloat16_rn(v); }

// Sum over the first `lanes` lanes, a power of two (the others get other sums).
__device__ __forceinline__ float lanes_sum(float v, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

// Largest of the warp's values that are numbers (NaN if none is).
__device__ __forceinline__ float warp_max(float v)
{
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// 4, 8 or 16 bytes read once, as W values.
template <int W, typename L>
__device__ __forceinline__ void load_values(const L *p, float *x)
{
    union {
        uint4 v4;
        uint2 v2;
        uint32_t v1;
        L one[16 / sizeof(L)];
    } u;
    if constexpr (W * sizeof(L) == 16) u.v4 = ld_stream_v4(p);
    else if constexpr (W * sizeof(L) == 8) u.v2 = ld_stream_v2(p);
    else if constexpr (W * sizeof(L) == 4) u.v1 = __ldg(reinterpret_cast<const uint32_t *>(p));
    else u.one[0] = *p;
#pragma unroll
    for (int i = 0; i < W; ++i) x[i] = to_float(u.one[i]);
}

template <int W, typename L>
__device__ __forceinline__ void store_values(L *p, const float *x)
{
    union {
        uint4 v4;
        uint2 v2;
        uint32_t v1;
        L one[16 / sizeof(L)];
    } u;
#pragma unroll
    for (int i = 0; i < W; ++i) u.one[i] = from_float(x[i], L());
    if constexpr (W * sizeof(L) == 16) st_v4(p, u.v4);
    else if constexpr (W * sizeof(L) == 8) st_v2(p, u.v2);
    else if constexpr (W * sizeof(L) == 4) *reinterpret_cast<uint32_t *>(p) = u.v1;
    else *p = u.one[0];
}

// Lane's NV logits of a row of E (-inf past E), W at a time: rows start on
// that many values' bytes, and E is a multiple of W.
template <int NV, int W, typename L>
__device__ __forceinline__ void load_row(const L *row, int E, int lane, float (&x)[NV])
{
#pragma unroll
    for (int j = 0; j < NV; ++j) x[j] = -INFINITY;
#pragma unroll
    for (int j = 0; j < NV; j += W)
        if (lane * NV + j < E) load_values<W>(row + lane * NV + j, x + j);
}

// Descending (no NaN among them), by Batcher's network of odd-even merges: 5,
// 19, 42 and 63 exchanges for 4, 8, 12 and 16 values.
template <int NV>
__device__ __forceinline__ void sort_values(float (&v)[NV])
{
#pragma unroll
    for (int p = 1; p < NV; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < NV; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < NV && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const float hi = fmaxf(v[i + j], v[i + j + k]), lo = fminf(v[i + j], v[i + j + k]);
                        v[i + j] = hi;
                        v[i + j + k] = lo;
                    }
}

template <int NV>
__device__ __forceinline__ float lane_max(const float (&x)[NV])
{
    float m = x[0];
#pragma unroll
    for (int j = 1; j < NV; ++j) m = fmaxf(m, x[j]);
    return m;
}

// The probability of logit x before the division by the row's sum: exactly 0
// at -inf, and NaN for NaN or +inf, which then reaches the whole row.  As a
// power of 2: the product's rounding grows with the distance to the maximum, a
// relative error of |x - m| 2^-24, and a power below 2^-126 is 0, where it would
// be subnormal: no sum here sees the difference.  Like the quotients by
// __fdividef (2 ulp) a choice for issue slots, within fp32's rounding: outputs
// of 16384 x 128 are within 7e-8 of 64 bits, PyTorch's fp32 operations 6e-8.
__device__ __forceinline__ float weight_of(float x, float m)
{
    return x == -INFINITY ? 0.0f : exp2_approx((x - m) * kLog2e);
}

// Whether rows of E values can be read (and written) `bytes` at a time.
bool rows_aligned(const void *p, const void *q, int E, int size, int bytes)
{
    return ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & (bytes - 1)) == 0 &&
           E * size % bytes == 0;
}

}  // namespace
}  // namespace moe

// Values a lane holds: the smallest of these that covers E, read in the widest
// loads that its rows' length and address allow.  12 are for fp32 alone, whose
// 16-byte load is 4 values; a bf16 one is 8, and E = 384 takes 16 values there
// (8192 tokens, K = 8: 21.9 us, fp32 16.4).
#define MOE_ROUTE_CASES(CALL, OTHER)                                            \
    if (bf16) {                                                                 \
        using L = __nv_bfloat16;                                                \
        if (E <= 128 && rows_aligned(logits, OTHER, E, 2, 8)) return CALL(4, 4, L);  \
        if (rows_aligned(logits, OTHER, E, 2, 16)) {                            \
            if (E <= 256) return CALL(8, 8, L);                                 \
            if (E <= 512) return CALL(16, 8, L);                                \
            return CALL(32, 8, L);                                              \
        }                                                                       \
        if (E <= 512 && rows_aligned(logits, OTHER, E, 2, 4)) {                 \
            if (E <= 256) return CALL(8, 2, L);                                 \
            return CALL(16, 2, L);                                              \
        }                                                                       \
        if (E <= 256) return CALL(8, 1, L);                                     \
        if (E <= 512) return CALL(16, 1, L);                                    \
        return CALL(32, 1, L);                                                  \
    }                                                                           \
    if (rows_aligned(logits, OTHER, E, 4, 16)) {                                \
        if (E <= 128) return CALL(4, 4, float);                                 \
        if (E <= 256) return CALL(8, 4, float);                                 \
        if (E <= 384) return CALL(12, 4, float);                                \
        if (E <= 512) return CALL(16, 4, float);                                \
        return CALL(32, 4, float);                                              \
    }                                                                           \
    if (E <= 128) return CALL(4, 1, float);                                     \
    if (E <= 256) return CALL(8, 1, float);                                     \
    if (E <= 512) return CALL(16, 1, float);                                    \
    return CALL(32, 1, float)
