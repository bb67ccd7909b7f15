// linear8.cuh -- kernels of the product of int8 matrices beside the one on the tensor cores
// (pair_gemm.cuh): few rows, and the sums of a split contraction.
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

// ------------------------------------------------------------------ few rows
// Bound by reading W once.  Each of a block's 8 warps takes 512 columns (16 bytes to a lane) of 4 k
// at a time: 4 x 4 bytes are turned round in registers, so that a word holds a column's 4 k, and
// multiplied with the row's 4 by one instruction (dp4a) into int32.  The contraction is split
// over the grid; int32 sums are exact in any order.
constexpr int BYTE_THREADS = 256, BYTE_ROWS = 8, BYTE_COLS = 512, BYTE_RANGE = 512, BYTE_STEP = 4;

struct ByteWork {
    int M, N, K;
    int across, ranges, range;   // range: a multiple of 32
    bool x_wide;
    int *partial;                // ranges x M x N
};

// Words a, b, c, d of four rows as words of four columns.
__device__ __forceinline__ void turn4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&out)[4]) {
    const uint32_t ab0 = __byte_perm(a, b, 0x5140), ab1 = __byte_perm(a, b, 0x7362);
    const uint32_t cd0 = __byte_perm(c, d, 0x5140), cd1 = __byte_perm(c, d, 0x7362);
    out[0] = __byte_perm(ab0, cd0, 0x5410), out[1] = __byte_perm(ab0, cd0, 0x7632);
    out[2] = __byte_perm(ab1, cd1, 0x5410), out[3] = __byte_perm(ab1, cd1, 0x7632);
}

template <int MR, bool WIDE>
__global__ void __launch_bounds__(BYTE_THREADS, MR <= 4 ? 2 : 1)
    byte_rows_kernel(ByteWork w, const signed char *X, long long ldx, const signed char *W, long long ldw) {
    constexpr int WARPS = BYTE_THREADS / 32;
    __shared__ __align__(16) int sums[BYTE_COLS * WARPS];
    __shared__ int xs[BYTE_RANGE / 4][MR];   // four k to a word
    sg::wait_prerequisites();
    sg::launch_dependents();
    const int n0 = (int(blockIdx.x) % w.across) * BYTE_COLS, q = int(blockIdx.x) / w.across;
    const int k0 = q * w.range, kn = min(w.range, w.K - k0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (!SG_IN_RANGE(kn > 0 && kn <= BYTE_RANGE && k0 + kn <= w.K && n0 < w.N && q < w.ranges && w.M <= MR)) return;
    for (int t = threadIdx.x; t < MR * ((kn + 3) / 4); t += BYTE_THREADS) {
        const int m = t % MR, k = t / MR * 4;
        uint32_t word = 0;
        if (m < w.M)
#pragma unroll
            for (int d = 0; d < 4; ++d)
                if (k + d < kn) word |= (uint32_t(X[m * ldx + k0 + k + d]) & 0xffu) << (8 * d);
        xs[k / 4][m] = int(word);
    }
    auto column = [&](int e) { return n0 + (WIDE ? lane * 16 + e : e * 32 + lane); };
    auto load = [&](int k) {   // 16 bytes of row k0 + k of W, zero past its end
        const signed char *p = W + (k0 + k) * ldw;
        if (k >= kn) return make_uint4(0, 0, 0, 0);
        if (WIDE && column(15) < w.N) return *reinterpret_cast<const uint4 *>(p + column(0));
        alignas(16) signed char v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = column(e) < w.N ? p[column(e)] : static_cast<signed char>(0);
        return *reinterpret_cast<const uint4 *>(v);
    };
    __syncthreads();
    int acc[MR][16] = {};
    for (int k = warp * (4 * BYTE_STEP); k < kn; k += WARPS * 4 * BYTE_STEP) {
        uint4 v[BYTE_STEP][4];
#pragma unroll
        for (int u = 0; u < BYTE_STEP; ++u)
#pragma unroll
            for (int d = 0; d < 4; ++d) v[u][d] = load(k + 4 * u + d);
#pragma unroll
        for (int u = 0; u < BYTE_STEP; ++u) {
            uint32_t c[4][4];
            turn4(v[u][0].x, v[u][1].x, v[u][2].x, v[u][3].x, c[0]);
            turn4(v[u][0].y, v[u][1].y, v[u][2].y, v[u][3].y, c[1]);
            turn4(v[u][0].z, v[u][1].z, v[u][2].z, v[u][3].z, c[2]);
            turn4(v[u][0].w, v[u][1].w, v[u][2].w, v[u][3].w, c[3]);
            if (k + 4 * u >= kn) break;
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                const int x = xs[(k + 4 * u) / 4][m];
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[m][e] = __dp4a(int(c[e / 4][e % 4]), x, acc[m][e]);
            }
        }
    }
    int *out = w.partial + (long long)q * w.M * w.N;
#pragma unroll
    for (int m = 0; m < MR; ++m) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 16; ++e) sums[warp * BYTE_COLS + (WIDE ? lane * 16 + e : e * 32 + lane)] = acc[m][e];
        __syncthreads();
        for (int t = threadIdx.x; t < BYTE_COLS; t += BYTE_THREADS) {
            int s = 0;
#pragma unroll
            for (int k = 0; k < WARPS; ++k) s += sums[k * BYTE_COLS + t];
            if (m < w.M && n0 + t < w.N) out[(long long)m * w.N + n0 + t] = s;
        }
    }
}

// ------------------------------------------------------------------ sums of ranges
// A thread to a column of a row, the ranges' sums and the scales (no range, K = 0: the bias, or 0).
template <class T>
__global__ void __launch_bounds__(256)
    byte_finish_kernel(int M, int N, int ranges, const int *__restrict__ partial, const float *scale, const float *wscale,
                       const T *bias, T *Y, long long ldy) {
    const int j = blockIdx.x * 256 + threadIdx.x;
    if (j >= N || !SG_IN_RANGE(int(blockIdx.y) < M)) return;
    if (ranges == 0) sg::wait_prerequisites();   // the call's only kernel: the inputs may just be being written
    const float of = ranges ? wscale[j] : 0.0f, b = bias ? to_f32(bias[j]) : 0.0f;
    sg::wait_prerequisites();
    const long long plane = (long long)M * N;
    for (long long i = blockIdx.y; i < M; i += gridDim.y) {
        int sum = 0;
#pragma unroll 8
        for (int r = 0; r < ranges; ++r) sum += partial[r * plane + i * N + j];
        const float v = ranges ? float(sum) * (scale[i] * of) : 0.0f;
        Y[i * ldy + j] = from_f32<T>(bias ? v + b : v);
    }
}

}  // namespace sgl
