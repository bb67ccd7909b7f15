// gate.cuh -- h = act(g) * u of the gated block, and its derivatives.
#pragma once

#include "activations.cuh"

namespace sgl {

// exp(-|z|): never over 1, so that neither form of the sigmoid below overflows or cancels.  bfloat16: by
// the approximate 2^x, whose argument's rounding makes it 8e-6 of itself off at |z| = 88, a
// thousandth of a rounding.
template <class T>
__device__ __forceinline__ float exp_minus(float z) {
    if constexpr (sizeof(T) == 4) return expf(-fabsf(z));
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(fabsf(z) * -1.44269504f));
    return y;
}
template <class T>
__device__ __forceinline__ float ratio(float a, float b) {   // b from 1 to 2
    if constexpr (sizeof(T) == 4) return __fdiv_rn(a, b);
    return a * reciprocal_fast(b);
}

// act(z) and act'(z).  SILU: z s, s + z s (1 - s) with s = 1 / (1 + exp(-z)), which is t / (1 + t) or
// 1 / (1 + t) by z's sign, t = exp(-|z|), and 1 - s the other one.
template <class T, int ACT>
__device__ __forceinline__ float2 gate_value(float2 z) {
    if constexpr (ACT == SGEMM_ACT_SILU) {
        const float tx = exp_minus<T>(z.x), ty = exp_minus<T>(z.y);
        return make_float2(z.x * ratio<T>(z.x < 0.0f ? tx : 1.0f, 1.0f + tx),
                           z.y * ratio<T>(z.y < 0.0f ? ty : 1.0f, 1.0f + ty));
    } else {
        return activate<T, ACT>(z);
    }
}
template <class T>
__device__ __forceinline__ void silu_both(float z, float &value, float &slope) {
    const float t = exp_minus<T>(z), one = ratio<T>(1.0f, 1.0f + t), other = t * one;
    const float s = z < 0.0f ? other : one, rest = z < 0.0f ? one : other;
    value = z * s;
    slope = fmaf(value, rest, s);
}
template <class T, int ACT>
__device__ __forceinline__ void gate_both(float2 z, float2 &value, float2 &rise) {
    if constexpr (ACT == SGEMM_ACT_SILU) {
        silu_both<T>(z.x, value.x, rise.x);
        silu_both<T>(z.y, value.y, rise.y);
    } else {
        value = activate<T, ACT>(z);
        rise = slope<T, ACT>(z);
    }
}

// f with the activation as a constant.
template <class F>
__device__ __forceinline__ void with_act(int act, F &&f) {
    switch (act) {
        case SGEMM_ACT_RELU: f(std::integral_constant<int, SGEMM_ACT_RELU>{}); break;
        case SGEMM_ACT_GELU: f(std::integral_constant<int, SGEMM_ACT_GELU>{}); break;
        case SGEMM_ACT_SILU: f(std::integral_constant<int, SGEMM_ACT_SILU>{}); break;
        default: f(std::integral_constant<int, SGEMM_ACT_NONE>{});
    }
}

}  // namespace sgl
