// activations.cuh -- the activations of sgemm_act and their derivatives, two elements at a time, to
// the accuracy of the element type T.
#pragma once

#include "../../include/sgemm_layers.h"
#include "elements.cuh"

namespace sgl {

// With Phi(z) = (1 + erf(z / sqrt 2)) / 2: tail = 1 - Phi(|z|) and bell = exp(-z^2/2).  tail /
// bell is a polynomial in a fraction of |z|; the exponential is the one that the derivative needs
// anyway, and both come without cancellation.
//
// bfloat16: formula 7.1.26 of Abramowitz and Stegun, Handbook of Mathematical Functions:
//   erf x = 1 - (a1 t + ... + a5 t^5) exp(-x^2),  t = 1 / (1 + p x),  x >= 0,
// whose error, at most 1.5e-7, is 1e-4 of a rounding here.  (x = |z| / sqrt 2 is folded into p,
// the half of Phi into the a's.)
//
// float32: tail / bell = (1 - v) Q(v) with v = 0.3 |z| / (1 + 0.3 |z|), Q of degree 9 fitted to the
// least relative error over |z| <= 14 (3.5e-9; with fp32's roundings 5e-7 of the tail, 4e-8 of 1).
// In v, not 1 - v, because then no rounding at z = 0 is magnified.  Against 64 bits GELU's
// gradient is 3.9e-8 off (2-norm; by 7.1.26 9.3e-8, by erff and expf 3.7e-8 but 199 us for 173 at
// 8192 x 16384), and small values at negative z keep their relative accuracy.
//
// Two elements at a time, and the approximate reciprocal alone for a division: GELU over 8192 x
// 16384 bfloat16 took 175 us one at a time, 126 with __fdividef.
__device__ __forceinline__ float exp2f_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float reciprocal_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

template <class T>
__device__ __forceinline__ void normal_tail(float2 z, float2 &tail, float2 &bell) {
    const float2 e = __fmul2_rn(__fmul2_rn(z, z), both(-0.72134752f));   // -z^2/2 log2 e
    bell = make_float2(exp2f_fast(e.x), exp2f_fast(e.y));
    if constexpr (sizeof(T) == 2) {
        const float2 t = make_float2(reciprocal_fast(fmaf(0.23164190f, fabsf(z.x), 1.0f)),
                                     reciprocal_fast(fmaf(0.23164190f, fabsf(z.y), 1.0f)));
        float2 p = __ffma2_rn(t, both(0.5307027145f), both(-0.7265760135f));
        p = __ffma2_rn(t, p, both(0.7107068705f));
        p = __ffma2_rn(t, p, both(-0.142248368f));
        p = __ffma2_rn(t, p, both(0.127414796f));
        tail = __fmul2_rn(__fmul2_rn(p, t), bell);
    } else {
        // (|z| of infinity is 64, where bell is 0: infinity times the reciprocal's 0 would be NaN)
        const float2 x = __fmul2_rn(make_float2(fminf(fabsf(z.x), 64.0f), fminf(fabsf(z.y), 64.0f)), both(0.3f));
        const float2 v = __fmul2_rn(x, make_float2(reciprocal_fast(1.0f + x.x), reciprocal_fast(1.0f + x.y)));
        float2 q = __ffma2_rn(v, both(0.0206178556f), both(-0.0731566458f));
        q = __ffma2_rn(v, q, both(0.0711469406f));
        q = __ffma2_rn(v, q, both(0.0101352528f));
        q = __ffma2_rn(v, q, both(0.0233557732f));
        q = __ffma2_rn(v, q, both(-0.139730486f));
        q = __ffma2_rn(v, q, both(-0.0810200348f));
        q = __ffma2_rn(v, q, both(0.618145186f));
        q = __ffma2_rn(v, q, both(-0.82980718f));
        q = __ffma2_rn(v, q, both(0.5f));
        tail = __fmul2_rn(__ffma2_rn(make_float2(-v.x, -v.y), q, q), bell);
    }
}

template <class T, int ACT>
__device__ __forceinline__ float2 activate(float2 z) {
    if constexpr (ACT == SGEMM_ACT_RELU)   // (a NaN stays one)
        return make_float2(z.x < 0.0f ? 0.0f : z.x, z.y < 0.0f ? 0.0f : z.y);
    // z Phi(z) = max(z, 0) - |z| tail, where +inf would be inf - inf * 0: its |z| is taken to be
    // the largest number.  (2 us of 115 at 8192 x 16384 bfloat16; a check of the result took 6.)
    if constexpr (ACT == SGEMM_ACT_GELU) {
        float2 tail, bell;
        normal_tail<T>(z, tail, bell);
        const float most = __uint_as_float(0x7f7fffffu);
        return make_float2(fmaf(-fabsf(fminf(z.x, most)), tail.x, fmaxf(z.x, 0.0f)),
                           fmaf(-fabsf(fminf(z.y, most)), tail.y, fmaxf(z.y, 0.0f)));
    }
    return z;
}

template <class T, int ACT>
__device__ __forceinline__ float2 slope(float2 z) {
    if constexpr (ACT == SGEMM_ACT_RELU)
        return make_float2(z.x > 0.0f ? 1.0f : (z.x <= 0.0f ? 0.0f : z.x),
                           z.y > 0.0f ? 1.0f : (z.y <= 0.0f ? 0.0f : z.y));
    if constexpr (ACT == SGEMM_ACT_GELU) {
        float2 tail, bell, cdf;
        normal_tail<T>(z, tail, bell);
        if constexpr (sizeof(T) == 2) {   // Phi(z) = 1/2 + sign(z) (1/2 - tail)
            const float2 h = __fadd2_rn(both(0.5f), make_float2(-tail.x, -tail.y));
            cdf = __fadd2_rn(both(0.5f), make_float2(copysignf(h.x, z.x), copysignf(h.y, z.y)));
        } else {                          // tail, or 1 - tail
            cdf = make_float2(z.x < 0.0f ? tail.x : 1.0f - tail.x, z.y < 0.0f ? tail.y : 1.0f - tail.y);
        }
        return __ffma2_rn(__fmul2_rn(z, both(0.39894228f)), bell, cdf);
    }
    return make_float2(z.x == z.x ? 1.0f : z.x, z.y == z.y ? 1.0f : z.y);
}

}  // namespace sgl
