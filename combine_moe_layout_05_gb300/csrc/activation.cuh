// activation.cuh -- the activations between the experts' products, and their
// slopes.  Each is z * sigmoid(u): u = z for SiLU; for GELU (its tanh form)
// u = 2 sqrt(2/pi) (z + 0.044715 z^3), since (1 + tanh v) / 2 = sigmoid(2 v).
//
// The sigmoid is one power of 2 and one reciprocal: a relative error of
// (1.3 |u| + 7) 2^-24, far below the bf16 rounding of what is made of it.  Below
// u = -88 it is 0, where the value itself is under 2^-126.
#pragma once

#include "common.cuh"
#include "moe_layout.h"

namespace moe {
namespace {

constexpr float kGelu = 1.5957691216057308f, kGeluCube = 0.044715f;

__device__ __forceinline__ float sigmoid_approx(float u) { return rcp_approx(1.0f + exp2_approx(-kLog2e * u)); }

__device__ __forceinline__ float gelu_argument(float z) { return z * fmaf(kGelu * kGeluCube, z * z, kGelu); }

__device__ __forceinline__ float silu(float z) { return z * sigmoid_approx(z); }
__device__ __forceinline__ float gelu(float z) { return z * sigmoid_approx(gelu_argument(z)); }

// d/dz of z * sigmoid(u(z)) = s + z s (1 - s) u'(z).
__device__ __forceinline__ float silu_slope(float z, float s) { return fmaf(z * s, 1.0f - s, s); }

// From |z| = 11 on s is 0 or 1, and so is the slope; z^2 stays finite, since 0
// times an infinity would be NaN (from 1.8e19 on).
__device__ __forceinline__ float gelu_slope(float z)
{
    const float s = sigmoid_approx(gelu_argument(z));
    return fmaf(z * s * (1.0f - s), fmaf(3.0f * kGelu * kGeluCube, fminf(z * z, 1e30f), kGelu), s);
}

}  // namespace
}  // namespace moe
