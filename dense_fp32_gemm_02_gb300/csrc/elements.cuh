// elements.cuh -- float32 and bfloat16 elements as the layer kernels read and
// write them: single elements, and eight consecutive ones as 16-byte accesses.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace sgl {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16 x) { return __bfloat162float(x); }

template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
    return x;
}
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float x) {
    return __float2bfloat16_rn(x);
}

// Division of u < 2^31 by an invariant d, in three instructions instead of about twenty
// (Granlund and Montgomery, Division by Invariant Integers using Multiplication, 1994).
struct Divisor {
    unsigned d, factor, shift;

    static Divisor of(unsigned d) {
        unsigned shift = 0;
        while ((1u << shift) < d) ++shift;
        const unsigned long long gap = (1ull << shift) - d;
        return Divisor{d, unsigned((gap << 32) / d + 1), shift};
    }
    __device__ unsigned quotient(unsigned u) const { return (__umulhi(u, factor) + u) >> shift; }
};

// The two bfloat16 of a 32-bit word (the lower address in the low half).
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Four consecutive elements, aligned to their size together.
__device__ __forceinline__ void load4(const float *p, float (&v)[4]) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}
__device__ __forceinline__ void load4(const bf16 *p, float (&v)[4]) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
}

__device__ __forceinline__ void store4(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(bf16 *p, const float (&v)[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

// Eight consecutive elements at a 16-byte aligned address.
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    const float4 b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16 *p, float (&v)[8]) {
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
    v[4] = bf16_lo(w.z), v[5] = bf16_hi(w.z), v[6] = bf16_lo(w.w), v[7] = bf16_hi(w.w);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(bf16 *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                               pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// The 4 N bytes from `shift` on of the 4 M in w, `shift` a multiple of GRAIN and at most 4 (M - N) - 1.
template <int GRAIN, int M, int N>
__device__ __forceinline__ void shift_bytes(uint32_t (&w)[M], int shift, uint32_t (&out)[N]) {
    static_assert(M == N + 1 || M == N + 2 || M == N + 4, "up to 3, 7 or 15 bytes");
    if (M == N + 4 && (shift & 8)) {
#pragma unroll
        for (int i = 0; i < N + 2; ++i) w[i] = w[i + 2];
    }
    if (M >= N + 2 && (shift & 4)) {
#pragma unroll
        for (int i = 0; i < (GRAIN == 4 ? N : N + 1); ++i) w[i] = w[i + 1];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = GRAIN == 4 ? w[i] : __funnelshift_r(w[i], w[i + 1], (shift & 3) * 8);
}

// Eight consecutive elements at any address, of a matrix from `begin` to `end`: the aligned 16 bytes that hold them,
// shifted into place (one by one they are eight accesses, of few bytes or 32 apart); false where those would leave the
// matrix.
template <class T>
__device__ __forceinline__ bool load8_shifted(const T *p, const T *begin, const T *end, float (&v)[8]) {
    constexpr int N = 2 * int(sizeof(T));
    const uintptr_t at = reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15);
    if (at < reinterpret_cast<uintptr_t>(begin) || at + 4 * N + 16 > reinterpret_cast<uintptr_t>(end)) return false;
    uint32_t w[N + 4], x[N];
#pragma unroll
    for (int i = 0; i < N + 4; i += 4) {
        const uint4 q = reinterpret_cast<const uint4 *>(at)[i / 4];
        w[i] = q.x, w[i + 1] = q.y, w[i + 2] = q.z, w[i + 3] = q.w;
    }
    shift_bytes<int(sizeof(T))>(w, int(reinterpret_cast<uintptr_t>(p) & 15), x);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = sizeof(T) == 4 ? __uint_as_float(x[i * N / 8]) : i & 1 ? bf16_hi(x[i / 2]) : bf16_lo(x[i / 2]);
    return true;
}

}  // namespace sgl
