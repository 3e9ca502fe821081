// The activations of a feed-forward block, and their derivatives, in FP32, two
// values at a time (packed arithmetic):
//
//   silu       x s(x)                s(u) = 1 / (1 + e^-u)
//   gelu       x Phi(x)              Phi the normal distribution
//   gelu_tanh  x (1 + tanh(v)) / 2 = x s(2 v),  v = sqrt(2 / pi) (x + 0.044715 x^3)
//
// e^x and 1 / x are the special-function unit's (2 ulp and 1 ulp).  An exponent
// of up to 58 rounded to FP32 moves its power more than that: silu is within
// 2^-18 of itself and gelu_tanh within 2^-17 where BF16 keeps 2^-9; below the
// clamps that follow they are within 2e-16 and 3e-15, but no longer of themselves.
// gelu is within 3e-7 |x|, and for x < 0 within 2^-14 of itself down to -12: Phi is
// 1 - Q(|x|), or Q for x < 0, Q = t (a1 + t (a2 + ... + t a6)) e^(-x^2 / 2),
// t = 1 / (1 + p |x|), whose seven numbers were fitted by linear programming to the
// least of the larger of |error| / 1e-7 and |error| / (2^-14 Q) on [0, 12]: 8e-8 and
// 4.1e-5 Q.  (Five terms, Hastings' in Abramowitz and Stegun 7.1.26, are as close but
// off by 0.16% of the value at -5 and 1% at -8, where BF16 rounds by 0.2% at most; the sixth
// costs 2 us of 398 at 8192 x 12288 x 4096.)
//
// The warps of a product's epilogue have nothing to hide this behind, so two
// values share one reciprocal, 1 / d0 = d1 (1 / (d0 d1)).  Hence x is held above
// -40 (silu) and -7 (gelu_tanh), where act is below 2e-16 and 3e-15 in magnitude,
// lest d0 d1 overflow; and a NaN is kept out of the reciprocal and meets its own
// result only, in the last operation.  The last bit of a value is then its
// neighbour's too, which may be a column beside it but not another row, of another
// token or of none: where the two are of different rows (OWN, the epilogue of few
// rows, which waits for memory: no slower) each has its own reciprocal.
// 8192 x 12288 x 4096: gelu adds 49 us to the product and silu 26; one value at a
// time they added 70 and 36.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rlk_internal.h"
#include "rlk_ptx.cuh"

namespace rlk {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluTwo = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 above(float2 x, float least) {
    return make_float2(fmax_nan(x.x, least), fmax_nan(x.y, least));
}
template <bool OWN>
__device__ __forceinline__ float2 rcp_pair(float2 d) {
    if (OWN) return make_float2(rcp_approx(d.x), rcp_approx(d.y));
    const float r = rcp_approx(d.x * d.y);
    return fmul2(make_float2(d.y, d.x), make_float2(r, r));
}

// e = 2^t and 1 / (1 + 2^t), t at most 58 where it is a number (the minimum takes
// that for a NaN).
template <bool OWN>
__device__ __forceinline__ float2 sigmoid_pair(float2 t, float2& e) {
    e = make_float2(ex2_approx(fminf(t.x, 58.f)), ex2_approx(fminf(t.y, 58.f)));
    return rcp_pair<OWN>(fadd2(e, both(1.f)));
}

// -Q(c) for c = min(|x|, 12), beyond which it is below 2e-33 (a NaN takes 12), and
// e^(-c^2 / 2).
template <bool OWN>
__device__ __forceinline__ float2 minus_tail_pair(float2 x, float2& c, float2& bell) {
    c = make_float2(fminf(fabsf(x.x), 12.f), fminf(fabsf(x.y), 12.f));
    const float2 t = rcp_pair<OWN>(ffma2(c, both(0.29249999f), both(1.f)));
    const float2 e = fmul2(fmul2(c, c), both(-0.5f * kLog2e));
    bell = make_float2(ex2_approx(e.x), ex2_approx(e.y));
    float2 p = ffma2(both(0.086254731f), t, both(-0.26742002f));
    p = ffma2(p, t, both(0.072400913f));
    p = ffma2(p, t, both(-0.16905613f));
    p = ffma2(p, t, both(-0.10457607f));
    p = ffma2(p, t, both(-0.11760336f));
    return fmul2(fmul2(p, t), bell);
}

// act of two values.
template <int ACT, bool OWN = false>
__device__ __forceinline__ float2 act_pair(float2 v) {
    if (ACT == RLK_ACT_RELU) return make_float2(v.x < 0.f ? 0.f : v.x, v.y < 0.f ? 0.f : v.y);
    if (ACT == RLK_ACT_SILU) {
        const float2 x = above(v, -40.f);
        float2 e;
        return fmul2(x, sigmoid_pair<OWN>(fmul2(x, both(-kLog2e)), e));
    }
    if (ACT == RLK_ACT_GELU_TANH) {
        const float2 x = above(v, -7.f);
        const float2 w = ffma2(fmul2(x, x), both(-kLog2e * kGeluTwo * kGeluCube), both(-kLog2e * kGeluTwo));
        float2 e;
        return fmul2(x, sigmoid_pair<OWN>(fmul2(x, w), e));
    }
    if (ACT == RLK_ACT_GELU) {  // x Phi(x) = max(x, 0) - |x| Q(|x|) for either sign
        float2 c, bell;
        const float2 tail = minus_tail_pair<OWN>(v, c, bell);
        return ffma2(c, tail, above(v, 0.f));
    }
    return v;
}

#define RLK_ACT_SWITCH(ACT, CALL)                         \
    switch (ACT) {                                        \
        case RLK_ACT_RELU: CALL(RLK_ACT_RELU) break;      \
        case RLK_ACT_SILU: CALL(RLK_ACT_SILU) break;      \
        case RLK_ACT_GELU: CALL(RLK_ACT_GELU) break;      \
        case RLK_ACT_GELU_TANH: CALL(RLK_ACT_GELU_TANH) break; \
        default: break;                                   \
    }

// act of the pairs [LO, HI) of v.
template <int LO, int HI, bool OWN = false, int N>
__device__ __forceinline__ void act_pairs(float2 (&v)[N], int act) {
#define RLK_ACT_ALL(A) _Pragma("unroll") for (int i = LO; i < HI; ++i) v[i] = act_pair<A, OWN>(v[i]);
    RLK_ACT_SWITCH(act, RLK_ACT_ALL)
#undef RLK_ACT_ALL
}

// act of one value, the same as of a pair of it.
__device__ __forceinline__ float act_one(float x, int act) {
    float2 v = both(x);
#define RLK_ACT_ONE(A) v = act_pair<A>(v);
    RLK_ACT_SWITCH(act, RLK_ACT_ONE)
#undef RLK_ACT_ONE
    return v.x;
}

// act'(x) of two values.  Beyond the clamps it is 0 or 1 to FP32, and within them
// no infinity meets a zero; a NaN stays one, and its neighbour does not.
template <int ACT>
__device__ __forceinline__ float2 act_slope_pair(float2 v) {
    constexpr float edge = ACT == RLK_ACT_SILU ? 40.f : ACT == RLK_ACT_GELU_TANH ? 7.f : 12.f;
    const float2 low = above(v, -edge);
    const float2 x = make_float2(fmin_nan(low.x, edge), fmin_nan(low.y, edge));
    if (ACT == RLK_ACT_SILU || ACT == RLK_ACT_GELU_TANH) {
        const float2 x2 = fmul2(x, x);
        // s = 1 / (1 + 2^t); x s' = x s (1 - s) u', u' = 1 (silu) or 2 sqrt(2 / pi) (1 + 3 . 0.044715 x^2)
        const float2 w = ACT == RLK_ACT_SILU ? both(-kLog2e)
                                             : ffma2(x2, both(-kLog2e * kGeluTwo * kGeluCube), both(-kLog2e * kGeluTwo));
        float2 e;
        const float2 s = sigmoid_pair<false>(fmul2(x, w), e);
        const float2 up = ACT == RLK_ACT_SILU ? both(1.f) : ffma2(x2, both(3.f * kGeluTwo * kGeluCube), both(kGeluTwo));
        // 1 - s is 2^t s, which keeps its digits where s is near 1 and x u' large
        return fmul2(s, ffma2(fmul2(x, up), fmul2(e, s), both(1.f)));
    }
    if (ACT == RLK_ACT_GELU) {
        float2 c, bell;
        const float2 h = fadd2(minus_tail_pair<false>(x, c, bell), both(0.5f));  // Phi(|x|) - 1/2
        const float2 p = fadd2(make_float2(copysignf(h.x, x.x), copysignf(h.y, x.y)), both(0.5f));
        return ffma2(fmul2(x, both(0.3989422804f)), bell, p);
    }
    return both(1.f);
}

// g act'(x).  relu passes g on or does not: an infinite g meets no zero.
template <int ACT>
__device__ __forceinline__ float2 act_back_pair(float2 g, float2 x) {
    if (ACT == RLK_ACT_RELU)
        return make_float2(x.x > 0.f ? g.x : x.x <= 0.f ? 0.f : x.x, x.y > 0.f ? g.y : x.y <= 0.f ? 0.f : x.y);
    return ACT == RLK_ACT_NONE ? g : fmul2(g, act_slope_pair<ACT>(x));
}

}  // namespace rlk
