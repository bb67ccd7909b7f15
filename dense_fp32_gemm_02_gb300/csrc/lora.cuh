// lora.cuh -- kernels of the adapter layer and of the weight gradient from a
// checkpoint.
#pragma once

#include "act8.cuh"
#include "adapters.cuh"
#include "kernels.cuh"

namespace sgl {

// A matrix read as fp32 elements: a row-major array, or a checkpoint.
template <class T>
struct Rows {
    const T *p;
    long long ld;
    __device__ float at(long long i, long long j) const { return to_f32(p[i * ld + j]); }
    __device__ void at8(long long i, long long j, float (&v)[8]) const { load8(p + i * ld + j, v); }
};
struct Act8Rows {
    const signed char *q, *e;
    long long ldq, lde;
    __device__ float at(long long i, long long j) const {
        return float(q[i * ldq + j]) * act8_step(e[i * lde + j / ACT8_BLOCK]);
    }
    __device__ void at8(long long i, long long j, float (&v)[8]) const {   // within a block
        const uint2 w = *reinterpret_cast<const uint2 *>(q + i * ldq + j);
        const float step = act8_step(e[i * lde + j / ACT8_BLOCK]);
        unpack_s8(w.x, v);
        unpack_s8(w.y, v + 4);
#pragma unroll
        for (int d = 0; d < 8; ++d) v[d] *= step;
    }
};

// ------------------------------------------------------------------ parts
// x as a sum of up to three bfloat16, each the leading 8 bits of what the ones before
// leave (cut, not rounded: x = x0 + x1 + x2 exactly, and no part overflows).  What is
// not finite stays in the first.
__device__ __forceinline__ void split_parts(float x, float (&part)[3]) {
    part[0] = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
    if ((__float_as_uint(x) & 0x7f800000u) == 0x7f800000u) {
        if (x != x) part[0] = __uint_as_float(0x7fc00000u);
        part[1] = part[2] = 0.0f;
        return;
    }
    const float rest = x - part[0];
    part[1] = __uint_as_float(__float_as_uint(rest) & 0xffff0000u);
    part[2] = rest - part[1];
}

// Where the parts of a matrix go: `planes` apart, rows `pitch` apart (both multiples
// of 8 elements, 16-byte aligned).
struct Parts {
    bf16 *p;
    long long pitch, plane;
};

// Eight consecutive elements of a row as PARTS planes.
template <int PARTS>
__device__ __forceinline__ void store_parts(const Parts &to, long long row, long long col,
                                            const float (&x)[8]) {
    float part[8][3];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (PARTS == 1) {
            part[i][0] = x[i];
        } else {
            split_parts(x[i], part[i]);
        }
    }
    bf16 *at = to.p + row * to.pitch + col;
#pragma unroll
    for (int q = 0; q < PARTS; ++q)
        *reinterpret_cast<uint4 *>(at + q * to.plane) =
            make_uint4(pack_bf16(part[0][q], part[1][q]), pack_bf16(part[2][q], part[3][q]),
                       pack_bf16(part[4][q], part[5][q]), pack_bf16(part[6][q], part[7][q]));
}

// The parts of a matrix: its values, a thread to eight columns.  One part suffices
// for bfloat16 (re-pitched for the TMA) and for a checkpoint.  `wide`: rows of X are
// 16-byte aligned (8-byte for a checkpoint's q).
template <int PARTS, class X>
__global__ void __launch_bounds__(256) parts_kernel(int M, int K, X x, bool wide, Parts to) {
    const int per_row = (K + 7) / 8;
    const long long total = (long long)M * per_row;
    for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < total;
         t += (long long)gridDim.x * 256) {
        const long long i = t / per_row;
        const int c = int(t - i * per_row) * 8;
        float v[8];
        if (wide && c + 8 <= K) {
            x.at8(i, c, v);
        } else {
#pragma unroll
            for (int d = 0; d < 8; ++d) v[d] = c + d < K ? x.at(i, c + d) : 0.0f;
        }
        store_parts<PARTS>(to, i, c, v);
    }
}

// ------------------------------------------------------------------ adapters of tiles
// For each 256 rows: the slot of the one adapter that all of them use, -1 where none
// of them uses any (or one of rank 0), -2 otherwise; slot_adapter lists the adapters of
// the slots in ascending order, -1 after them.  One block.
constexpr int MAX_ADAPTERS = 1024;

__global__ void __launch_bounds__(1024)
    tile_adapters_kernel(int M, int tiles, int slots, Adapters ad, int *tile_adapter, int *slot_adapter) {
    __shared__ int slot_of[MAX_ADAPTERS];
    __shared__ int warp_sum[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    slot_of[threadIdx.x] = 0;
    __syncthreads();
    for (int t = warp; t < tiles; t += 32) {
        const long long r0 = (long long)t * 256;
        int a = ad.of_row(r0);
        bool same = true;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const long long r = r0 + i * 32 + lane;
            if (r < M) same = same && ad.of_row(r) == a;
        }
        same = __all_sync(0xffffffffu, same);
        if (lane == 0) {
            if (same && a >= 0 && ad.rank(a) == 0) a = -1;
            tile_adapter[t] = same ? a : -2;
            if (same && a >= 0) slot_of[a] = 1;
        }
    }
    __syncthreads();
    // slots in ascending order of the adapters: a prefix sum over the flags
    const int flag = slot_of[threadIdx.x];
    int sum = flag;
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < 32; ++w) {
        before += w < warp ? warp_sum[w] : 0;
        all += warp_sum[w];
    }
    const int slot = before + sum - flag;
    slot_of[threadIdx.x] = slot;
    if (flag && SG_IN_RANGE(slot < slots)) slot_adapter[slot] = threadIdx.x;
    for (int s = all + threadIdx.x; s < slots; s += 1024) slot_adapter[s] = -1;
    __syncthreads();
    for (int t = threadIdx.x; t < tiles; t += 1024) {
        const int a = tile_adapter[t];
        if (a >= 0) tile_adapter[t] = slot_of[a];
    }
}

// The parts of the slots' adapters, planes part * slots + slot of rows x cols, zero
// past the adapter's rank (RANK_ROWS: the rank runs down the rows, else along them).
template <class T, bool RANK_ROWS>
__global__ void __launch_bounds__(256)
    pack_stack_kernel(int rows, int cols, Stack<const T> V, Adapters ad, const int *slot_adapter,
                      int slots, Parts to) {
    constexpr int PARTS = sizeof(T) == 4 ? 3 : 1;
    const int slot = blockIdx.y, a = slot_adapter[slot];
    if (a < 0) return;
    const int rank = ad.rank(a), per_row = (cols + 7) / 8;
    const T *v = V.matrix(a);
    Parts at = to;
    at.p += slot * to.plane;
    at.plane = to.plane * slots;
    const long long total = (long long)rows * per_row;
    for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < total;
         t += (long long)gridDim.x * 256) {
        const long long i = t / per_row;
        const int c = int(t - i * per_row) * 8;
        float x[8];
#pragma unroll
        for (int d = 0; d < 8; ++d)
            x[d] = (c + d < cols && (RANK_ROWS ? i : c + d) < rank) ? to_f32(v[i * V.ld + c + d]) : 0.0f;
        store_parts<PARTS>(at, i, c, x);
    }
}

// ------------------------------------------------------------------ rank side
// What the rank-side product of a direction leaves behind: S (M x R, scaled), the same
// as parts where `parts.p` is not null, and unscaled for the caller in H.
struct RankSide {
    float *S;
    long long lds;
    float *H;
    long long ldh;
    Parts parts;
};

// S[i][r] = scale * sum_c X[i][c] * V_a[c][r] for the rows that use an adapter, 0
// elsewhere: a warp to an (i, r) pair.  TRANS: V_a is stored R x C.
template <class T, bool TRANS>
__global__ void __launch_bounds__(256)
    rank_side_kernel(int M, int C, Rows<T> X, Stack<const T> V, Adapters ad, RankSide to) {
    const int lane = threadIdx.x & 31;
    const long long pair = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const long long i = pair / ad.R;
    const int r = int(pair - i * ad.R);
    if (i >= M) return;
    const int a = ad.of_row(i);
    float sum = 0.0f, scaled = 0.0f;
    if (a >= 0 && r < ad.rank(a)) {
        const T *v = V.matrix(a);
        for (int c = lane; c < C; c += 32)
            sum = fmaf(X.at(i, c), to_f32(TRANS ? v[r * V.ld + c] : v[c * V.ld + r]), sum);
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        scaled = sum * ad.scale(a);
    }
    if (lane != 0) return;
    if (to.H) to.H[i * to.ldh + r] = sum;
    to.S[i * to.lds + r] = scaled;
    if (to.parts.p) {
        float part[3];
        split_parts(scaled, part);
        for (int q = 0; q < (sizeof(T) == 4 ? 3 : 2); ++q)
            to.parts.p[q * to.parts.plane + i * to.parts.pitch + r] = __float2bfloat16_rn(part[q]);
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
