// rows.cuh -- the adapter layer for few rows (a decode step): Y = X W + bias + rank side.
//
// Bound by reading W once (and of the stack what the rows use).  W goes through shared
// memory by asynchronous copies, 128 columns of a range of K to a block, three slabs
// ahead; the warp-level MMA takes the rows 16 at a time, so that 1 row and 16 cost the
// same.  In the same launch, blocks of their own take the rank side row by row, each row
// with its own adapter.  A second kernel adds the ranges in order and applies the rest.
#pragma once

#include "rank_products.cuh"

namespace sgl {

constexpr int FEW_ROWS = 64, ROWS_COLS = 128;

template <class T, int MT>
struct FewRows {
    static constexpr bool F32 = sizeof(T) == 4;
    static constexpr int PARTS = F32 ? 3 : 1, STAGES = 4;
    static constexpr int W_PITCH = ROWS_COLS + (F32 ? 4 : 8), W_ELEMS = SLAB * W_PITCH;
    static constexpr int X_PITCH = SLAB + 8, X_PLANE = MT * 16 * X_PITCH;
    static constexpr size_t SMEM = size_t(STAGES) * W_ELEMS * sizeof(T) + size_t(2) * PARTS * X_PLANE * 2;
};

// The work of a launch: `across` x `ranges` blocks of the product, then M x `rank_ranges`
// blocks of the rank side.
struct RowsWork {
    int M, N, K;
    int across, ranges, range;
    int rank_ranges, rank_range;
    float *partial;        // ranges x M x N
    float *rank_partial;   // rank_ranges x M x R
};

// The rank side of one row over one range: threads along the rank and, in groups, along
// the range, whose sums are added in order.
template <class T>
__device__ __forceinline__ void rank_of_row(const RowsWork &w, int b, const Rows<T> &X, const Stack<const T> &V,
                                            const Adapters &ad, float *sums) {
    const int i = b / w.rank_ranges, q = b - i * w.rank_ranges;
    const int a = ad.of_row(i);
    const int rank = a < 0 ? 0 : ad.rank(a);
    if (rank == 0) return;   // nothing reads this row's sums
    const int width = ad.R <= 8 ? 8 : ad.R <= 16 ? 16 : ad.R <= 32 ? 32 : ad.R <= 64 ? 64 : 128;
    const int groups = RANK_THREADS / width, r = threadIdx.x & (width - 1), group = threadIdx.x / width;
    const int c1 = min(w.K, (q + 1) * w.rank_range);
    const T *x = X.p + i * X.ld, *v = V.matrix(a) + r;
    float sum = 0.0f;
    if (r < rank) {
#pragma unroll 8
        for (int c = q * w.rank_range + group; c < c1; c += groups)
            sum = fmaf(to_f32(x[c]), to_f32(v[c * V.ld]), sum);
    }
    sums[threadIdx.x] = sum;
    __syncthreads();
    if (group == 0 && r < rank) {
        for (int g = 1; g < groups; ++g) sum += sums[g * width + r];
        w.rank_partial[((long long)q * w.M + i) * ad.R + r] = sum;
    }
}

template <class T, int MT>
__global__ void __launch_bounds__(RANK_THREADS)
    few_rows_kernel(RowsWork w, Rows<T> X, const T *W, long long ldw, bool w_wide, Stack<const T> V, Adapters ad) {
    using Z = FewRows<T, MT>;
    constexpr int PARTS = Z::PARTS, STAGES = Z::STAGES;
    extern __shared__ __align__(16) unsigned char smem_rows[];
    if (int(blockIdx.x) >= w.across * w.ranges) {
        rank_of_row(w, int(blockIdx.x) - w.across * w.ranges, X, V, ad, reinterpret_cast<float *>(smem_rows));
        return;
    }
    T *ring = reinterpret_cast<T *>(smem_rows);
    bf16 *xs = reinterpret_cast<bf16 *>(ring + STAGES * Z::W_ELEMS);   // [2][PARTS][16 MT rows]
    const int n0 = (int(blockIdx.x) % w.across) * ROWS_COLS, q = int(blockIdx.x) / w.across;
    const int k_begin = q * w.range, k_end = min(w.K, k_begin + w.range);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    auto fill = [&](int stage, int k0) {
        T *ws = ring + stage * Z::W_ELEMS;
        constexpr int PER = 16 / int(sizeof(T)), ALONG = ROWS_COLS / PER;
#pragma unroll
        for (int o = threadIdx.x; o < SLAB * ALONG; o += RANK_THREADS) {
            const int k = o / ALONG, c = (o % ALONG) * PER;
            const bool in = k0 + k < k_end && n0 + c < w.N;
            fill16(ws + k * Z::W_PITCH + c, in ? W + (k0 + k) * ldw + n0 + c : W, in ? w.N - n0 - c : 0, w_wide);
        }
    };
    // a slab of X, 16 MT x 64, as parts: MT * 4 elements to a thread, four at a time
    float xv[MT][4];
    auto load_x = [&](int k0) {
#pragma unroll
        for (int h = 0; h < MT; ++h) {
            const int o = threadIdx.x + h * RANK_THREADS, m = o / 16, k = k0 + (o % 16) * 4;
#pragma unroll
            for (int d = 0; d < 4; ++d) xv[h][d] = m < w.M && k + d < k_end ? X.at(m, k + d) : 0.0f;
        }
    };
    auto stage_x = [&](bf16 *to) {
#pragma unroll
        for (int h = 0; h < MT; ++h) {
            const int o = threadIdx.x + h * RANK_THREADS, m = o / 16, k = (o % 16) * 4;
            uint32_t lo[3], hi[3];
            pair_parts(xv[h][0], xv[h][1], lo);
            pair_parts(xv[h][2], xv[h][3], hi);
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
                *reinterpret_cast<uint2 *>(to + p * Z::X_PLANE + m * Z::X_PITCH + k) =
                    PARTS == 1 ? make_uint2(pack_bf16(xv[h][0], xv[h][1]), pack_bf16(xv[h][2], xv[h][3]))
                               : make_uint2(lo[p], hi[p]);
        }
    };

    float sum[MT][2][4] = {};
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
        if (k_begin + s * SLAB < k_end) fill(s, k_begin + s * SLAB);
        sg::cp_async_commit();
    }
    load_x(k_begin);
    int stage = 0;
    for (int k0 = k_begin; k0 < k_end; k0 += SLAB) {
        bf16 *x = xs + (stage & 1) * PARTS * Z::X_PLANE;
        stage_x(x);
        sg::cp_async_wait<STAGES - 2>();
        __syncthreads();   // this slab has landed, and the stage filled next has been read
        if (k0 + (STAGES - 1) * SLAB < k_end) fill((stage + STAGES - 1) % STAGES, k0 + (STAGES - 1) * SLAB);
        sg::cp_async_commit();
        if (k0 + SLAB < k_end) load_x(k0 + SLAB);
        const T *ws = ring + stage * Z::W_ELEMS;
        float big[MT][2][4] = {}, small[MT][2][4] = {};
#pragma unroll
        for (int kk = 0; kk < SLAB; kk += 16) {
            uint32_t fb[PARTS][4];   // two 8-column tiles of 16 k
            if constexpr (!Z::F32) {
                ldmatrix4<true>(fb[0], ws + (kk + (lane & 15)) * Z::W_PITCH + warp * 16 + ((lane >> 4) & 1) * 8);
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const T *p = ws + (kk + (lane & 3) * 2 + (d & 1) * 8) * Z::W_PITCH + warp * 16 + (lane >> 2) + (d >> 1) * 8;
                    uint32_t part[3];
                    pair_parts(p[0], p[Z::W_PITCH], part);
                    fb[0][d] = part[0], fb[1][d] = part[1], fb[2][d] = part[2];
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int pa = PARTS - 1; pa >= 0; --pa) {
                    uint32_t fa[4];
                    ldmatrix4<false>(fa, x + pa * Z::X_PLANE + (m * 16 + (lane & 15)) * Z::X_PITCH + kk + (lane >> 4) * 8);
#pragma unroll
                    for (int pb = 0; pb < PARTS - pa; ++pb)
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            mma16816(pa + pb > 0 ? small[m][t] : big[m][t], fa, fb[pb][2 * t], fb[pb][2 * t + 1]);
                }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    sum[m][t][d] += Z::F32 ? big[m][t][d] + small[m][t][d] : big[m][t][d];
        stage = (stage + 1) % STAGES;
    }
    float *out = w.partial + (long long)q * w.M * w.N;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int i = m * 16 + (lane >> 2) + (d / 2) * 8, j = n0 + warp * 16 + t * 8 + (lane & 3) * 2 + (d & 1);
                if (i < w.M && j < w.N) out[(long long)i * w.N + j] = sum[m][t][d];
            }
}

// Y from the partial sums: a block to 256 columns of a row.  The first one of a row also
// writes H.
template <class T>
__global__ void __launch_bounds__(256)
    few_rows_finish_kernel(RowsWork w, Stack<const T> V, Adapters ad, const T *bias, float *H, long long ldh, T *Y,
                           long long ldy) {
    __shared__ float S[128];
    const int i = blockIdx.y, j = blockIdx.x * 256 + threadIdx.x;
    const int a = ad.of_row(i), rank = a < 0 ? 0 : ad.rank(a);
    if (int(threadIdx.x) < ad.R && ad.L > 0) {
        const int r = threadIdx.x;
        float sum = 0.0f;
        if (r < rank)
            for (int q = 0; q < w.rank_ranges; ++q) sum += w.rank_partial[((long long)q * w.M + i) * ad.R + r];
        if (H && blockIdx.x == 0) H[i * ldh + r] = sum;
        S[r] = r < rank ? sum * ad.scale(a) : 0.0f;
    }
    __syncthreads();
    if (j >= w.N) return;
    float x = 0.0f;
    const float *p = w.partial + (long long)i * w.N + j;
    const long long plane = (long long)w.M * w.N;
#pragma unroll 8
    for (int q = 0; q < w.ranges; ++q) x += p[q * plane];
    if (bias) x += to_f32(bias[j]);
    if (rank > 0) {
        const T *v = V.matrix(a) + j;
#pragma unroll 8
        for (int r = 0; r < rank; ++r) x = fmaf(S[r], to_f32(v[r * V.ld]), x);
    }
    Y[(long long)i * ldy + j] = from_f32<T>(x);
}

}  // namespace sgl
