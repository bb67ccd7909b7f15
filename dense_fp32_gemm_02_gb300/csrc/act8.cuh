// act8.cuh -- the 8-bit form of an activation matrix: one exponent e for each
// block of 32 columns of a row, x ~ q * 2^e with q in int8.
//
// The step is a power of two, so x / 2^e and q * 2^e are exact in fp32 (the
// rounding of q is the only one), and q * 2^e, of at most 7 significant bits, is
// exact in bfloat16: a product with a checkpoint takes it as one bfloat16
// operand without rounding it again.  A step of t/127 would be up to twice
// finer (1.4 times on average) and have neither property.
#pragma once

#include "elements.cuh"

namespace sgl {

constexpr int ACT8_BLOCK = 32;
constexpr int ACT8_NAN = -128;   // the exponent of a block that holds an infinity or a NaN

__device__ __forceinline__ uint32_t magnitude_bits(float x) {
    return __float_as_uint(x) & 0x7fffffffu;
}

// The exponent of a block from the bits of its largest magnitude t: the least
// e >= -126 with t <= 127 * 2^e, and 121 where that is 122 (127 * 2^122 is past
// fp32: q then stops at 127).  Magnitudes order as their bits do.  With t =
// 1.f * 2^E, 127 * 2^(E-6) = 1.984375 * 2^E decides between E - 6 and E - 5.
__device__ __forceinline__ int act8_exponent(uint32_t top) {
    if (top >= 0x7f800000u) return ACT8_NAN;
    const int E = int(top >> 23) - 127;
    return min(max(E - 6 + ((top & 0x7fffffu) > 0x7e0000u ? 1 : 0), -126), 121);
}

// 2^-e for an exponent other than ACT8_NAN (a normal number).
__device__ __forceinline__ float act8_inverse_step(int e) {
    return __uint_as_float(uint32_t(127 - e) << 23);
}
// q of an element, given 2^-e.
__device__ __forceinline__ int act8_quantise(float x, float inverse_step) {
    return max(-127, min(127, __float2int_rn(x * inverse_step)));
}
// 2^e, or NaN for ACT8_NAN.
__device__ __forceinline__ float act8_step(int e) {
    return e == ACT8_NAN ? __uint_as_float(0x7fc00000u) : __uint_as_float(uint32_t(e + 127) << 23);
}

// Conversions between int8 and float by way of the low bits of a float of known exponent:
// the converting instructions run at a quarter of the rate of these.
//
// Four int8 of a word as floats: 2^23 + (q + 128) by its bytes, less 2^23 + 128.
__device__ __forceinline__ void unpack_s8(uint32_t w, float *v) {
    w ^= 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540u + i)) - 8388736.0f;
}
// Four values of at most 127 in magnitude after scaling, rounded to nearest even, as the
// bytes of a word: 1.5 * 2^23 + x keeps the integer in its low bits.
__device__ __forceinline__ uint32_t pack_s8(const float *x, float scale) {
    const float2 s = make_float2(scale, scale), magic = make_float2(12582912.0f, 12582912.0f);
    const float2 a = __ffma2_rn(make_float2(x[0], x[1]), s, magic);
    const float2 b = __ffma2_rn(make_float2(x[2], x[3]), s, magic);
    return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                       __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
}

}  // namespace sgl
