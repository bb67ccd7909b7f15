// linear8.cuh -- the product of int8 matrices beside its kernels on the tensor cores (byte_tiles.cuh, and
// pair_gemm.cuh for many rows): bytes as operands, and the sums of a split contraction.
//
//   y_ij = scale_i * wscale_j * sum_k q_ik w_kj + bias_j,   the sum exact in int32
#pragma once

#include "lora.cuh"

namespace sgl {

// A matrix of int8 as PartsJob reads it: its values are bfloat16 as they are.
struct ByteRows {
    const signed char *p;
    long long ld;
    __device__ float at(long long i, long long j) const { return float(p[i * ld + j]); }
    __device__ void at8(long long i, long long j, float (&v)[8]) const {
        const uint2 w = *reinterpret_cast<const uint2 *>(p + i * ld + j);
        unpack_s8(w.x, v);
        unpack_s8(w.y, v + 4);
    }
};

// ------------------------------------------------------------------ sums of ranges
// A thread to four columns of a row, the ranges' sums and the scales (no range, K = 0: the bias, or 0).
template <class T>
__global__ void __launch_bounds__(128)
    byte_finish_kernel(int M, int N, int ranges, const int *__restrict__ partial, const float *scale, const float *wscale,
                       const T *bias, T *Y, long long ldy) {
    const int j = (blockIdx.x * 128 + threadIdx.x) * 4, n = min(4, N - j);
    if (j >= N || !SG_IN_RANGE(int(blockIdx.y) < M)) return;
    if (ranges == 0) sg::wait_prerequisites();   // the call's only kernel: the inputs may just be being written
    float of[4], b[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        of[d] = ranges && d < n ? wscale[j + d] : 0.0f;
        b[d] = bias && d < n ? to_f32(bias[j + d]) : 0.0f;
    }
    sg::wait_prerequisites();
    const long long plane = (long long)M * N;
    for (long long i = blockIdx.y; i < M; i += gridDim.y) {
        int sum[4] = {};
        const int *p = partial + i * N + j;
        if (N % 4 == 0) {
#pragma unroll 8
            for (int r = 0; r < ranges; ++r) {
                const int4 v = *reinterpret_cast<const int4 *>(p + r * plane);
                sum[0] += v.x, sum[1] += v.y, sum[2] += v.z, sum[3] += v.w;
            }
        } else {
#pragma unroll 4
            for (int r = 0; r < ranges; ++r)
#pragma unroll
                for (int d = 0; d < 4; ++d) sum[d] += d < n ? p[r * plane + d] : 0;
        }
        const float row = ranges ? scale[i] : 0.0f;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const float v = ranges ? float(sum[d]) * (row * of[d]) : 0.0f;
            if (d < n) Y[i * ldy + j + d] = from_f32<T>(bias ? v + b[d] : v);
        }
    }
}

}  // namespace sgl
