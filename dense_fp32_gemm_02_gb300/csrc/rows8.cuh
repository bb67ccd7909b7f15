// rows8.cuh -- a row in 8 bits: scale = max|p| / 127, q = rint(127 p / max|p|), exactly rounded.
//
// 127 p / max is worked out in fp32 (at most 4 roundings, 3.1e-5 in q's units), and where that is within
// NEAR = 2^-14 of a tie the products are compared exactly.
#pragma once

#include "act8.cuh"

namespace sgl {

constexpr float NEAR = 0x1p-14f;
// The range of the largest |p| in which fp32 products and 127 / max lose nothing; rows outside it
// are quantised in 64 bits.
constexpr float LEAST_TOP = 0x1p-60f, MOST_TOP = 0x1p100f;

// To an integer: 1.5 * 2^23 leaves no fraction.
__device__ __forceinline__ float whole(float quotient) { return (quotient + 12582912.0f) - 12582912.0f; }

// q of |p| near a tie: n or n + 1, n the whole part of the fp32 quotient, by the sign of 127 |p| - (n
// + 1/2) top.  p of 24 bits (from bfloat16 16): the difference of the products in fp32 is exact, as it
// is under 2^18 units of p's last place, and so is what (n + 1/2) top leaves.  (In bfloat16 ties are no
// rare thing: a row whose largest value is 127 / 32 has 32 x for a quotient.)
__device__ __forceinline__ float tie_exact(float p, float quotient, float top) {
    const float n = floorf(fabsf(quotient)), h = n + 0.5f, t = h * top;
    const float d = fmaf(127.0f, fabsf(p), -t) - fmaf(h, top, -t);
    const bool odd = (int(n) & 1) != 0;
    return copysignf(d > 0.0f || (d == 0.0f && odd) ? n + 1.0f : n, quotient);
}

}  // namespace sgl
