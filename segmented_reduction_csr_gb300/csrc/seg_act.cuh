// seg_act.cuh -- the activations of the gated block and their derivatives, in float32.
#pragma once
#include "seg_gated.cuh"

namespace segred {

// s(x) = 1 / (1 + exp(-x)) and s(-x) = 1 - s(x), from exp(-|x|) so that neither
// overflows nor cancels.  FAST: the special function unit's exponential, off by 2 +
// 1.2 |x| units of 2^-23, and quotient, off by 2; else 3 units in all.
template <bool FAST>
__device__ __forceinline__ void logistic(float x, float& s, float& other) {
    const float e = FAST ? __expf(-fabsf(x)) : expf(-fabsf(x));
    const float high = FAST ? __fdividef(1.0f, 1.0f + e) : 1.0f / (1.0f + e), low = e * high;
    // (NaN: both are)
    s = x >= 0.0f ? high : low;
    other = x >= 0.0f ? low : high;
}

// The normal distribution below -|x|, as exp(-x^2 / 2) t poly(t), t = 1 / (1 + 0.33
// |x| / sqrt(2)): the form of Hastings (Approximations for Digital Computers,
// 1955), its coefficients fitted to the whole tail at once (the fit's largest
// relative error is 1.2e-7 in exact arithmetic; erfcf took twice the instructions).
// In float32, in units of 2^-23: the exponential 2 + 1.7 x^2 / 2 with its argument's
// rounding, t 3, which t poly(t) passes on 3.5 times, the polynomial's roundings 3,
// its fit 1, the products 2: below 23 + 0.85 x^2.  e: exp(-x^2 / 2).
__device__ __forceinline__ float normal_tail(float x, float& e) {
    e = __expf(-0.5f * x * x);
    const float t = __fdividef(1.0f, fmaf(0.23334524f, fabsf(x), 1.0f));
    float s = -0.13534459f;
    s = fmaf(s, t, 0.46023273f);
    s = fmaf(s, t, -0.35114244f);
    s = fmaf(s, t, 0.40849352f);
    s = fmaf(s, t, 0.04722397f);
    s = fmaf(s, t, 0.20122291f);
    s = fmaf(s, t, 0.18295610f);
    s = fmaf(s, t, 0.18635780f);
    return 0.5f * s * t * e;
}

// act(x) and, where `slope` is wanted, act'(x).
//   silu      x s                       s + x s (1 - s)            s = logistic(x)
//   gelu      x P                       P + x p                    P, p: the normal distribution and its density
//   gelu_tanh x s                       s + x s (1 - s) q'         s = logistic(q) = (1 + tanh(q / 2)) / 2,
//                                                                  q = sqrt(8 / pi) (x + 0.044715 x^3)
//   relu      max(x, 0)                 1 where x > 0, else 0
//   sigmoid   s                         s (1 - s)
// Off by, in units of 2^-23 at most (exponents by their own roundings too: 3 |q| for
// gelu_tanh): FAST silu, sigmoid 4 + 1.2 |x|, gelu_tanh 4 + 4.2 |q|, gelu 23 + 0.85
// x^2, and results below 2^-121 may be 0; else 3.5, 3.5 + 3 |q| and 6 + 1.1 x^2.
template <bool FAST, bool SLOPE>
__device__ __forceinline__ float activate(int kind, float x, float& slope) {
    if (kind == ACT_RELU) {
        // (NaN stays NaN)
        if (SLOPE) slope = x > 0.0f ? 1.0f : 0.0f;
        return x > 0.0f || x != x ? x : 0.0f;
    }
    if (kind == ACT_GELU) {
        float p, e;
        if (FAST) {
            p = normal_tail(x, e);
            if (x > 0.0f) p = 1.0f - p;
        } else {
            p = 0.5f * erfcf(-0.70710678f * x);
            if (SLOPE) e = expf(-0.5f * x * x);
        }
        if (SLOPE) {
            slope = e > 0.0f ? fmaf(x, 0.39894228f * e, p) : p;
        }
        return x * p;
    }
    float q = x, dq = 1.0f;
    if (kind == ACT_GELU_TANH) {
        const float x2 = fminf(x * x, 1e6f);      // (s is 0 or 1 long before that)
        q = 1.5957691f * x * fmaf(0.044715f, x2, 1.0f);
        if (SLOPE) dq = 1.5957691f * fmaf(0.134145f, x2, 1.0f);
    }
    if constexpr (FAST && !SLOPE) {
        // s alone: exp(-q) may overflow, 1 / inf is 0
        float r;
        asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-q)));
        return kind == ACT_SIGMOID ? r : x * r;
    }
    float s, other;
    logistic<FAST>(q, s, other);
    const float f = kind == ACT_SIGMOID ? s : x * s;
    if (SLOPE) {
        const float rest = s * other;
        // (x may be so large that its product with 0 is none)
        slope = kind == ACT_SIGMOID ? rest : rest > 0.0f ? fmaf(x * dq, rest, s) : s;
    }
    return f;
}

}  // namespace segred
