// The activations of a feed-forward block, and their derivatives, in FP32.
//
//   silu       x s(x)                s(u) = 1 / (1 + e^-u)
//   gelu       x Phi(x)              Phi the normal distribution
//   gelu_tanh  x (1 + tanh(v)) / 2 = x s(2 v),  v = sqrt(2 / pi) (x + 0.044715 x^3)
//
// e^x is the special-function unit's (2 ulp) and so is 1 / x (1 ulp): 2^-21 of
// the result, where BF16 keeps 2^-9.  Phi is 1 - erfc(|x| / sqrt 2) / 2 (or
// the second term for x < 0) with the five-term approximation of erfc by
// Hastings (Abramowitz and Stegun 7.1.26): t (a1 + t (a2 + ...)) e^-y^2 with
// t = 1 / (1 + p y), within 1.5e-7 of erfc, so 7.5e-8 of Phi, about one FP32
// rounding of 1.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rlk_internal.h"
#include "rlk_ptx.cuh"

namespace rlk {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluTwo = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;

__device__ __forceinline__ float sigmoid_f32(float u) { return rcp_approx(1.f + ex2_approx(-kLog2e * u)); }

// Phi(x), and e^(-x^2 / 2) with it.
__device__ __forceinline__ float normal_cdf(float x, float& bell) {
    const float y = fabsf(x) * 0.70710678f, t = rcp_approx(__fmaf_rn(0.3275911f, y, 1.f));
    bell = ex2_approx(x * x * (-0.5f * kLog2e));
    float p = __fmaf_rn(1.061405429f, t, -1.453152027f);
    p = __fmaf_rn(p, t, 1.421413741f);
    p = __fmaf_rn(p, t, -0.284496736f);
    p = __fmaf_rn(p, t, 0.254829592f);
    const float half = 0.5f * p * t * bell;  // erfc / 2
    return x < 0.f ? half : 1.f - half;
}

// act(x); NaN stays NaN.
__device__ __forceinline__ float act_f32(float x, int act) {
    switch (act) {
        case RLK_ACT_RELU: return x < 0.f ? 0.f : x;
        case RLK_ACT_SILU: return x * sigmoid_f32(x);
        case RLK_ACT_GELU: {
            float bell;
            return x * normal_cdf(x, bell);
        }
        case RLK_ACT_GELU_TANH: return x * sigmoid_f32(kGeluTwo * x * __fmaf_rn(kGeluCube, x * x, 1.f));
        default: return x;
    }
}

// act'(x).  Beyond +-20 the derivative is 0 or 1 to FP32 (silu: +-90); x is
// kept within, so that no infinity meets a zero.
__device__ __forceinline__ float act_slope_f32(float x, int act) {
    const float edge = act == RLK_ACT_SILU ? 90.f : 20.f;
    const float y = x > edge ? edge : x < -edge ? -edge : x;
    switch (act) {
        case RLK_ACT_RELU: return x > 0.f ? 1.f : x <= 0.f ? 0.f : x;
        case RLK_ACT_SILU: {
            const float s = sigmoid_f32(y);
            return s * __fmaf_rn(y, 1.f - s, 1.f);
        }
        case RLK_ACT_GELU: {
            float bell;
            const float p = normal_cdf(y, bell);
            return __fmaf_rn(0.3989422804f * y, bell, p);
        }
        case RLK_ACT_GELU_TANH: {
            const float s = sigmoid_f32(kGeluTwo * y * __fmaf_rn(kGeluCube, y * y, 1.f));
            return __fmaf_rn(y * s * (1.f - s) * kGeluTwo, __fmaf_rn(3.f * kGeluCube, y * y, 1.f), s);
        }
        default: return 1.f;
    }
}

}  // namespace rlk
