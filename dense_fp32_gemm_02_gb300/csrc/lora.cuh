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

// ------------------------------------------------------------------ rows by adapter
// Rows grouped by their adapter, in the order of the rows within a group (a stable
// counting sort), and the work lists of the kernels that walk the groups.  Rows
// without an adapter, or with one of rank 0, come last, as group L.
struct Groups {
    int *perm;           // M: row numbers, group after group
    int *totals;         // {tiles, chunks}
    int4 *tiles;         // of up to ROW_TILE rows: {adapter or -1, first place in perm, rows, 0}
    int4 *chunks;        // of up to `chunk` rows of an adapter: the same
    int *chunk_begin;    // L + 1: the chunks of adapter a are [a], .. [a + 1]
    int chunk;
    int *tile_adapter;   // for each 256 rows of the call: see Product (may be null)
    int *slot_adapter;   // `slots` of them, in ascending order, -1 after the last
    int slots;
};
constexpr int MAX_ADAPTERS = 1024, ROW_TILE = 64, SORT_THREADS = 1024;

// Exclusive prefix sum over one value per thread of a 1024-thread block; `all` their sum.
__device__ __forceinline__ int block_prefix(int v, int *warp_sum, int &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int sum = v;
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    int before = 0;
    all = 0;
    for (int w = 0; w < 32; ++w) {
        before += w < warp ? warp_sum[w] : 0;
        all += warp_sum[w];
    }
    return before + sum - v;
}

// The group of place `t` given the groups' first places (n + 1 of them, ascending).
__device__ __forceinline__ int group_at(const int *first, int n, int t) {
    int lo = 0, hi = n;   // first[lo] <= t < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        (first[mid] <= t ? lo : hi) = mid;
    }
    return lo;
}

constexpr size_t sort_smem(int L) { return (size_t(32) * (L + 1) + 3 * (L + 2)) * 4; }

// One block: M is tens of thousands of rows at most in practice, and each warp walks
// its share of them twice.
__global__ void __launch_bounds__(SORT_THREADS, 1)
    group_rows_kernel(int M, Adapters ad, Groups g) {
    extern __shared__ int sm[];
    __shared__ int warp_sum[32];
    const int L = ad.L, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int *count = sm;                       // [warp][group], then the next place of each
    int *first = count + 32 * (L + 1);     // L + 2: first place of a group
    int *tile0 = first + (L + 2), *chunk0 = tile0 + (L + 2);
    for (int i = threadIdx.x; i < 32 * (L + 1); i += SORT_THREADS) count[i] = 0;
    __syncthreads();
    const long long per = ((M + 31LL) / 32 + 31) / 32 * 32;
    const long long r0 = warp * per, r1 = min(r0 + per, (long long)M);
    auto group_of = [&](long long r) {
        const int a = ad.of_row(r);
        return a < 0 || ad.rank(a) == 0 ? L : a;
    };
    int *mine = count + warp * (L + 1);
    for (long long r = r0; r < r1; r += 32) {
        const bool in = r + lane < r1;
        const int a = in ? group_of(r + lane) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, a);
        if (in && (same & ((1u << lane) - 1)) == 0) mine[a] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // first places of the groups (up to 1025 of them: group L by the last thread alone)
    int rows = 0, all;
    const int a = threadIdx.x;
    if (a < L)
        for (int w = 0; w < 32; ++w) rows += count[w * (L + 1) + a];
    const int at = block_prefix(rows, warp_sum, all);
    const int tile_at = block_prefix((rows + ROW_TILE - 1) / ROW_TILE, warp_sum, all);
    if (a < L) first[a] = at, tile0[a] = tile_at;
    if (a == SORT_THREADS - 1) {
        first[L] = at + rows;
        tile0[L] = all;
        first[L + 1] = M;
        tile0[L + 1] = all + (M - first[L] + ROW_TILE - 1) / ROW_TILE;
    }
    const int chunk_at = block_prefix((rows + g.chunk - 1) / g.chunk, warp_sum, all);
    if (a < L) chunk0[a] = chunk_at;
    if (a == SORT_THREADS - 1) chunk0[L] = all;
    __syncthreads();
    for (int b = threadIdx.x; b <= L; b += SORT_THREADS) {
        g.chunk_begin[b] = chunk0[b];
        int place = first[b];
        for (int w = 0; w < 32; ++w) {
            const int n = count[w * (L + 1) + b];
            count[w * (L + 1) + b] = place;
            place += n;
        }
    }
    if (threadIdx.x == 0) g.totals[0] = tile0[L + 1], g.totals[1] = chunk0[L];
    __syncthreads();
    for (long long r = r0; r < r1; r += 32) {
        const bool in = r + lane < r1;
        const int b = in ? group_of(r + lane) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, b);
        const int before = __popc(same & ((1u << lane) - 1));
        const int place = in ? mine[b] + before : 0;
        __syncwarp();
        if (in && SG_IN_RANGE(place >= 0 && place < M)) g.perm[place] = int(r + lane);
        if (in && before == 0) mine[b] += __popc(same);
        __syncwarp();
    }
    for (int t = threadIdx.x; t < tile0[L + 1]; t += SORT_THREADS) {
        const int b = group_at(tile0, L + 1, t), p = first[b] + (t - tile0[b]) * ROW_TILE;
        g.tiles[t] = make_int4(b < L ? b : -1, p, min(ROW_TILE, first[b + 1] - p), 0);
    }
    for (int t = threadIdx.x; t < chunk0[L]; t += SORT_THREADS) {
        const int b = group_at(chunk0, L, t), p = first[b] + (t - chunk0[b]) * g.chunk;
        g.chunks[t] = make_int4(b, p, min(g.chunk, first[b + 1] - p), 0);
    }
    if (!g.tile_adapter) return;
    // tiles of 256 rows with one adapter, and the slots of those adapters
    int *flag = count;
    __syncthreads();
    flag[min(int(threadIdx.x), 32 * (L + 1) - 1)] = 0;
    __syncthreads();
    const int tiles = (M + 255) / 256;
    for (int t = warp; t < tiles; t += 32) {
        const long long q0 = (long long)t * 256;
        const int b = group_of(q0);
        bool same = true;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const long long r = q0 + i * 32 + lane;
            if (r < M) same = same && group_of(r) == b;
        }
        same = __all_sync(0xffffffffu, same);
        if (lane == 0) {
            g.tile_adapter[t] = !same ? -2 : (b < L ? b : -1);
            if (same && b < L) flag[b] = 1;
        }
    }
    __syncthreads();
    const int used = a < L ? flag[a] : 0;
    const int slot = block_prefix(used, warp_sum, all);
    if (used && SG_IN_RANGE(slot < g.slots)) g.slot_adapter[slot] = a;
    if (a < L) flag[a] = slot;
    for (int s = all + threadIdx.x; s < g.slots; s += SORT_THREADS) g.slot_adapter[s] = -1;
    __syncthreads();
    for (int t = threadIdx.x; t < tiles; t += SORT_THREADS) {
        const int b = g.tile_adapter[t];
        if (b >= 0) g.tile_adapter[t] = flag[b];
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

}  // namespace sgl
