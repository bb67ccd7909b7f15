// lora.cuh -- kernels of the adapter layer and of the weight gradient from a
// checkpoint.
#pragma once

#include "act8.cuh"

namespace sgl {

// The adapters of a call: which one a row uses, its rank and scale.
struct Adapters {
    const int *ids, *ranks;
    const float *scales;
    int L, R;

    __device__ int of_row(long long i) const {
        const int a = L > 0 ? ids[i] : -1;
        return unsigned(a) < unsigned(L) ? a : -1;
    }
    __device__ int rank(int a) const { return ranks ? min(max(ranks[a], 0), R) : R; }
    __device__ float scale(int a) const { return scales ? scales[a] : 1.0f; }
};

// A stack of L matrices.
template <class T>
struct Stack {
    T *p;
    long long ld, stride;

    __device__ T *matrix(int a) const { return p + a * stride; }
};

// A matrix read as fp32 elements: (row, column) of a row-major array, of its
// transpose, or of a checkpoint.
template <class T>
struct Rows {
    const T *p;
    long long ld;
    __device__ float at(long long i, long long j) const { return to_f32(p[i * ld + j]); }
};
template <class T>
struct Transposed {
    const T *p;
    long long ld;
    __device__ float at(long long i, long long j) const { return to_f32(p[j * ld + i]); }
};
struct Act8Rows {
    const signed char *q, *e;
    long long ldq, lde;
    __device__ float at(long long i, long long j) const {
        return float(q[i * ldq + j]) * act8_step(e[i * lde + j / ACT8_BLOCK]);
    }
};
struct Act8Transposed {
    Act8Rows x;
    __device__ float at(long long i, long long j) const { return x.at(j, i); }
};

// S[i][r] = factor * sum_c X[i][c] * V_a[c][r] for the rows that use an adapter,
// 0 elsewhere: a warp to an (i, r) pair.  TRANS: V_a is stored R x C.
template <class T, bool TRANS>
__global__ void __launch_bounds__(256)
    rank_side_kernel(int M, int C, Rows<T> X, Stack<const T> V, Adapters ad, bool scaled, float *S,
                     long long lds) {
    const int lane = threadIdx.x & 31;
    const long long pair = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const long long i = pair / ad.R;
    const int r = int(pair - i * ad.R);
    if (i >= M) return;
    const int a = ad.of_row(i);
    float sum = 0.0f;
    if (a >= 0 && r < ad.rank(a)) {
        const T *v = V.matrix(a);
        for (int c = lane; c < C; c += 32)
            sum = fmaf(X.at(i, c), to_f32(TRANS ? v[r * V.ld + c] : v[c * V.ld + r]), sum);
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (scaled) sum *= ad.scale(a);
    }
    if (lane == 0) S[i * lds + r] = sum;
}

// The rank-side term of an output element: sum_r S[i][r] * V_a, by fp32 FMAs
// over the ranks of the row's own adapter only.
template <class T, bool TRANS>
struct Expand {
    Adapters ad;
    const float *S;
    long long lds;
    Stack<const T> V;
    bool scaled;

    __device__ float at(long long i, long long j) const {
        const int a = ad.of_row(i);
        if (a < 0) return 0.0f;
        const int rank = ad.rank(a);
        const T *v = V.matrix(a);
        float sum = 0.0f;
        for (int r = 0; r < rank; ++r)
            sum = fmaf(S[i * lds + r], to_f32(TRANS ? v[j * V.ld + r] : v[r * V.ld + j]), sum);
        return scaled ? sum * ad.scale(a) : sum;
    }
};
struct NoExpand {
    __device__ float at(long long, long long) const { return 0.0f; }
};

// out = P * Q + expand + bias + beta * out, 64 x 64 tiles, 4 x 4 to a thread.
template <class T, class PA, class QB, class E>
__global__ void __launch_bounds__(256)
    product_kernel(int M, int N, int K, PA P, QB Q, E expand, const T *bias, float beta, T *out,
                   long long ldo) {
    __shared__ float p[16][65], q[16][65];
    const long long i0 = (long long)blockIdx.y * 64, j0 = (long long)blockIdx.x * 64;
    const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += 16) {
        for (int t = threadIdx.x; t < 16 * 64; t += 256) {
            const int k = t / 64, x = t % 64;
            p[k][x] = (i0 + x < M && k0 + k < K) ? P.at(i0 + x, k0 + k) : 0.0f;
            q[k][x] = (j0 + x < N && k0 + k < K) ? Q.at(k0 + k, j0 + x) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < 16; ++k)
            for (int y = 0; y < 4; ++y)
                for (int x = 0; x < 4; ++x)
                    acc[y][x] = fmaf(p[k][ti + 16 * y], q[k][tj + 16 * x], acc[y][x]);
        __syncthreads();
    }
    for (int y = 0; y < 4; ++y)
        for (int x = 0; x < 4; ++x) {
            const long long i = i0 + ti + 16 * y, j = j0 + tj + 16 * x;
            if (i >= M || j >= N) continue;
            float v = acc[y][x] + expand.at(i, j);
            if (bias) v += to_f32(bias[j]);
            if (beta != 0.0f) v = fmaf(beta, to_f32(out[i * ldo + j]), v);
            out[i * ldo + j] = from_f32<T>(v);
        }
}

// The gradients of a stack: out_a[c][r] = sum over the rows i of a of
// factor * X[i][c] * S[i][r] (TRANS: stored R x C): a thread to an element.
template <class T, bool TRANS, class XR>
__global__ void __launch_bounds__(256)
    stack_grad_kernel(int M, int C, XR X, const float *S, long long lds, Adapters ad, bool scaled,
                      Stack<T> out) {
    const int c = blockIdx.x * 256 + threadIdx.x, r = blockIdx.y, a = blockIdx.z;
    if (c >= C) return;
    float sum = 0.0f;
    if (r < ad.rank(a)) {
        for (int i = 0; i < M; ++i)
            if (ad.of_row(i) == a) sum = fmaf(X.at(i, c), S[i * lds + r], sum);
        if (scaled) sum *= ad.scale(a);
    }
    out.matrix(a)[TRANS ? r * out.ld + c : c * out.ld + r] = from_f32<T>(sum);
}

}  // namespace sgl
