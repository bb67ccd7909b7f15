// linear8.cuh -- the product of int8 matrices beside its kernels on the tensor cores (byte_tiles.cuh, and
// pair_gemm.cuh for many rows): bytes as operands, and the sums of a split contraction.
//
//   y_ij = scale_i * wscale_j * sum_k q_ik w_kj + bias_j,   the sum exact in int32
#pragma once

#include "lora.cuh"

namespace sgl {

// ------------------------------------------------------------------ bytes as operands
// Rows of int8 as rows of bfloat16, which hold them as they are, for pair_gemm.cuh.  A warp to 2048
// columns of a row.  X's kernel sets `large` to 1 if the magnitudes of such a piece add up to more than
// 2^17: with W's at most 2^7, a sum of 2048 products may then leave the 2^24 that fp32 holds exactly.
// W's kernel, which comes first, sets it to 0; X's runs beside it and waits before that one write.  (Rows
// that the call has brought to 8 bits itself were complete before W's kernel let X's start.)
constexpr int BYTE_PIECE = 2048;
constexpr unsigned MOST_MAGNITUDES = 131072;

struct ByteJob {
    const signed char *p;
    long long ld;
    int rows, cols;
    Parts to;
    bool wide;       // rows are 8-byte aligned

    __host__ __device__ int pieces() const { return (cols + BYTE_PIECE - 1) / BYTE_PIECE; }
    __host__ __device__ long long items() const { return (long long)rows * pieces(); }
};

// (the piece's magnitudes added up, where SUM)
template <bool SUM>
__device__ __forceinline__ unsigned take_bytes(const ByteJob &job, long long item) {
    const int lane = threadIdx.x & 31, pieces = job.pieces();
    const long long row = item / pieces;
    const int c0 = int(item - row * pieces) * BYTE_PIECE;
    if (!SG_IN_RANGE(row < job.rows && c0 < job.cols)) return 0;
    const signed char *from = job.p + row * job.ld;
    bf16 *to = job.to.p + row * job.to.pitch;
    uint2 v[BYTE_PIECE / 256];   // eight columns to a lane, so that what is written is whole lines too
#pragma unroll
    for (int i = 0; i < BYTE_PIECE / 256; ++i) {
        const int c = c0 + i * 256 + lane * 8;
        v[i] = make_uint2(0, 0);
        if (job.wide && c + 8 <= job.cols) {
            v[i] = *reinterpret_cast<const uint2 *>(from + c);
        } else if (c < job.cols) {
            alignas(8) signed char x[8];
#pragma unroll
            for (int d = 0; d < 8; ++d) x[d] = c + d < job.cols ? from[c + d] : static_cast<signed char>(0);
            v[i] = *reinterpret_cast<const uint2 *>(x);
        }
    }
    unsigned sum = 0;
#pragma unroll
    for (int i = 0; i < BYTE_PIECE / 256; ++i) {
        const int c = c0 + i * 256 + lane * 8;
        const uint32_t w[2] = {v[i].x, v[i].y};
        float f[8];
        unpack_s8(w[0], f);
        unpack_s8(w[1], f + 4);
        if (SUM) {
#pragma unroll
            for (int d = 0; d < 2; ++d) {   // |q| is q or ~q + 1, byte by byte
                const uint32_t sign = w[d] >> 7 & 0x01010101u;
                sum = __dp4a((w[d] ^ (sign * 0xffu)), 0x01010101u, __dp4a(sign, 0x01010101u, sum));
            }
        }
        if (c < job.cols)   // (the pitch is a multiple of 8)
            *reinterpret_cast<uint4 *>(to + c) = make_uint4(pack_exact(f[0], f[1]), pack_exact(f[2], f[3]),
                                                            pack_exact(f[4], f[5]), pack_exact(f[6], f[7]));
    }
    return SUM ? __reduce_add_sync(0xffffffffu, sum) : 0;
}

template <bool ROWS>   // X's rows; else W
__global__ void __launch_bounds__(256) byte_expand_kernel(ByteJob job, int *large) {
    if (!ROWS) sg::wait_prerequisites();
    sg::launch_dependents();
    if (!ROWS && blockIdx.x == 0 && threadIdx.x == 0) *large = 0;
    const long long warps = (long long)gridDim.x * 8, total = job.items();
    bool over = false;
    for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += warps)
        over |= take_bytes<ROWS>(job, i) > MOST_MAGNITUDES;
    if (!ROWS) return;
    sg::wait_prerequisites();
    if (over && (threadIdx.x & 31) == 0) atomicExch(large, 1);
}

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
