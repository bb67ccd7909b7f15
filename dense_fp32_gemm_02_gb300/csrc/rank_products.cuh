// rank_products.cuh -- the two skinny products of the adapter layer, over rows grouped
// by adapter: the rank side, S = X * V_a (rows of a group x R), and the gradients of
// the stack, X^T * S over the rows of a group (C x R).
//
// One side of each is at most 128 wide, so both are bound by reading X once (R = 16:
// 16 flop per byte of bfloat16), and their rows lie anywhere in X.  So the warp-level
// MMA (m16n8k16, bfloat16, fp32 accumulators) is fast enough: its operands come from
// shared memory that plain loads fill row by row, from any alignment, converting on
// the way: a float32 element as three bfloat16 parts, a checkpoint's as one (see
// parts_gemm.cuh for the parts).
//
// A block only ever holds rows of one adapter, and of its stack the columns below its
// rank: nothing of another adapter is multiplied, not even by zero.
//
// The MMA's additions truncate, so a slab's products (64 of the contraction; the small
// pairs of parts first) add up from zero and then go to fp32 sums, round to nearest:
// four additions of full size to a slab truncate, 5e-7 at most.
#pragma once

#include "lora.cuh"

namespace sgl {

constexpr int SLAB = 64;              // of the contraction
constexpr int RANK_THREADS = 256;
constexpr int PITCH64 = SLAB + 8;     // elements: rows 16 bytes past a multiple of 128

__device__ __forceinline__ uint32_t shared_address(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
template <bool TRANSPOSE>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
    if constexpr (TRANSPOSE)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Eight elements as PARTS planes of shared memory, `plane` elements apart.
template <int PARTS>
__device__ __forceinline__ void stage8(bf16 *to, int plane, const float (&x)[8]) {
    store_parts<PARTS>(Parts{to, 0, plane}, 0, 0, x);
}

// What the rank side leaves behind: S (M x R, scaled), the same as parts where
// `parts.p` is not null, and unscaled for the caller in H.
struct RankSide {
    float *S;
    long long lds;
    float *H;
    long long ldh;
    Parts parts;

    template <class T>
    __device__ void put(long long i, int r, float sum, float scale) const {
        if (H) H[i * ldh + r] = sum;
        const float s = sum * scale;
        S[i * lds + r] = s;
        if (parts.p) {
            float part[3];
            split_parts(s, part);
            // (bfloat16: two parts, 2^-16, under the output's rounding)
            for (int q = 0; q < (sizeof(T) == 4 ? 3 : 2); ++q)
                parts.p[q * parts.plane + i * parts.pitch + r] = __float2bfloat16_rn(part[q]);
        }
    }
};

// S of one tile of up to 64 rows of a group (blockIdx.x) over one range of the
// contraction (blockIdx.y): 8 warps, 16 rows x half of the rank each.  NT: the rank in
// units of 8, rounded up to 2, 4, 8 or 16.  TRANS: V_a is stored R x C.  With one
// range the results go to `to`, otherwise to partial[range][row][R].
template <class T, bool TRANS, int NT>
struct RankTile {
    static constexpr int PARTS = sizeof(T) == 4 ? 3 : 1, WN = NT / 2, RP = NT * 8;
    static constexpr int X_PLANE = ROW_TILE * PITCH64;
    static constexpr int V_ROWS = TRANS ? RP : SLAB, V_PITCH = TRANS ? PITCH64 : RP + 8;
    static constexpr int V_PLANE = V_ROWS * V_PITCH;
    static constexpr size_t SMEM = size_t(PARTS) * (X_PLANE + V_PLANE) * 2;
};

template <class T, bool TRANS, int NT>
__global__ void __launch_bounds__(RANK_THREADS)
    rank_tile_kernel(int C, int range, Rows<T> X, bool x_wide, Stack<const T> V, bool v_wide, Adapters ad,
                     Groups g, float *partial, long long partial_plane, RankSide to) {
    using Z = RankTile<T, TRANS, NT>;
    constexpr int PARTS = Z::PARTS, WN = Z::WN;
    constexpr int VO = Z::V_ROWS * (TRANS ? SLAB : Z::RP) / 8;            // octets of the V slab
    constexpr int VN = (VO + RANK_THREADS - 1) / RANK_THREADS;
    extern __shared__ __align__(16) unsigned char smem_rank[];
    bf16 *xs = reinterpret_cast<bf16 *>(smem_rank), *vs = xs + PARTS * Z::X_PLANE;
    __shared__ int rows[ROW_TILE];
    if (int(blockIdx.x) >= g.totals[0]) return;
    const int4 tile = g.tiles[blockIdx.x];
    const int a = tile.x, n = tile.z;
    if (threadIdx.x < ROW_TILE) rows[threadIdx.x] = int(threadIdx.x) < n ? g.perm[tile.y + threadIdx.x] : -1;
    __syncthreads();
    if (a < 0) {   // rows without an adapter: only the caller's H shows them
        if (to.H && blockIdx.y == 0)
            for (int t = threadIdx.x; t < n * ad.R; t += RANK_THREADS)
                to.H[(long long)rows[t / ad.R] * to.ldh + t % ad.R] = 0.0f;
        return;
    }
    const int rank = ad.rank(a);
    const T *v = V.matrix(a);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wm = warp & 3, wn = warp >> 2;
    const int c_begin = blockIdx.y * range, c_end = min(C, c_begin + range);

    float xv[2][8], vv[VN][8];
    auto load = [&](int c0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {   // 64 rows x 8 octets
            const int o = threadIdx.x + h * RANK_THREADS, i = rows[o / 8], c = c0 + (o % 8) * 8;
            if (i >= 0 && x_wide && c + 8 <= c_end) {
                X.at8(i, c, xv[h]);
            } else {
#pragma unroll
                for (int d = 0; d < 8; ++d) xv[h][d] = (i >= 0 && c + d < c_end) ? X.at(i, c + d) : 0.0f;
            }
        }
#pragma unroll
        for (int h = 0; h < VN; ++h) {
            const int o = threadIdx.x + h * RANK_THREADS;
            if (VO % RANK_THREADS != 0 && o >= VO) break;
            constexpr int PER = (TRANS ? SLAB : Z::RP) / 8;
            const int row = o / PER, col = (o % PER) * 8;
            // (TRANS: row is r and col c - c0; else row is c - c0 and col r)
            const int cs = TRANS ? c0 + col : c0 + row, r = TRANS ? row : col;
            const T *p = v + (TRANS ? (long long)r * V.ld + cs : (long long)cs * V.ld + r);
            const bool whole = TRANS ? r < rank && cs + 8 <= c_end : r + 8 <= rank && cs < c_end;
            if (whole && v_wide) {
                load8(p, vv[h]);
            } else {
#pragma unroll
                for (int d = 0; d < 8; ++d)
                    vv[h][d] = (TRANS ? r < rank && cs + d < c_end : r + d < rank && cs < c_end) ? to_f32(p[d]) : 0.0f;
            }
        }
    };

    float sum[WN][4] = {};
    load(c_begin);
    for (int c0 = c_begin; c0 < c_end; c0 += SLAB) {
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int o = threadIdx.x + h * RANK_THREADS;
            stage8<PARTS>(xs + (o / 8) * PITCH64 + (o % 8) * 8, Z::X_PLANE, xv[h]);
        }
#pragma unroll
        for (int h = 0; h < VN; ++h) {
            const int o = threadIdx.x + h * RANK_THREADS;
            if (VO % RANK_THREADS != 0 && o >= VO) break;
            constexpr int PER = (TRANS ? SLAB : Z::RP) / 8;
            stage8<PARTS>(vs + (o / PER) * Z::V_PITCH + (o % PER) * 8, Z::V_PLANE, vv[h]);
        }
        __syncthreads();
        if (c0 + SLAB < c_end) load(c0 + SLAB);
        float acc[WN][4] = {};
        auto products = [&](int qa, int qb) {
#pragma unroll
            for (int kk = 0; kk < SLAB; kk += 16) {
                uint32_t fa[4];
                ldmatrix4<false>(fa, shared_address(xs + qa * Z::X_PLANE + (wm * 16 + (lane & 15)) * PITCH64 + kk +
                                                    (lane >> 4) * 8));
#pragma unroll
                for (int t = 0; t < WN; t += 2) {
                    const int n0 = (wn * WN + t) * 8;
                    uint32_t fb[4];
                    const bf16 *at = vs + qb * Z::V_PLANE;
                    if constexpr (TRANS)
                        at += (n0 + (lane & 7) + (WN > 1 ? ((lane >> 4) & 1) * 8 : 0)) * PITCH64 + kk + ((lane >> 3) & 1) * 8;
                    else
                        at += (kk + (lane & 15)) * Z::V_PITCH + n0 + (WN > 1 ? ((lane >> 4) & 1) * 8 : 0);
                    ldmatrix4<!TRANS>(fb, shared_address(at));
                    mma16816(acc[t], fa, fb[0], fb[1]);
                    if constexpr (WN > 1) mma16816(acc[t + 1], fa, fb[2], fb[3]);
                }
            }
        };
        if constexpr (PARTS == 3) {
            products(0, 2), products(2, 0), products(1, 1), products(0, 1), products(1, 0);
        }
        products(0, 0);
#pragma unroll
        for (int t = 0; t < WN; ++t)
#pragma unroll
            for (int d = 0; d < 4; ++d) sum[t][d] += acc[t][d];
    }
    const float scale = ad.scale(a);
#pragma unroll
    for (int t = 0; t < WN; ++t)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int m = wm * 16 + (lane >> 2) + (d / 2) * 8, r = (wn * WN + t) * 8 + (lane & 3) * 2 + (d & 1);
            if (m >= n || r >= ad.R) continue;
            const long long i = rows[m];
            if (gridDim.y > 1)
                partial[blockIdx.y * partial_plane + i * ad.R + r] = sum[t][d];
            else
                to.put<T>(i, r, sum[t][d], scale);
        }
}

// The ranges' partial sums of the rank side, added in order.
template <class T>
__global__ void __launch_bounds__(256)
    rank_finish_kernel(int M, int ranges, const float *__restrict__ partial, long long plane, Adapters ad,
                       RankSide to) {
    const long long total = (long long)M * ad.R;
    for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < total; t += (long long)gridDim.x * 256) {
        const long long i = t / ad.R;
        const int a = ad.of_row(i);
        if (a < 0 || ad.rank(a) == 0) continue;
        float sum = 0.0f;
#pragma unroll 8
        for (int s = 0; s < ranges; ++s) sum += partial[s * plane + t];
        to.put<T>(i, int(t - i * ad.R), sum, ad.scale(a));
    }
}

// X^T * S over a chunk of rows of a group (blockIdx.y), 128 columns of X (blockIdx.x):
// 8 warps, 16 columns x the whole rank each.  partial[chunk] is C x R, or R x C where
// RANK_ROWS.  S (and whether it still is to be scaled) as the rank side left it.
template <class X, int PA, int PB, int NT>
struct StackTile {
    static constexpr int COLS = 128, X_PITCH = COLS + 8, S_PITCH = NT * 8 + 8;
    static constexpr int X_PLANE = SLAB * X_PITCH, S_PLANE = SLAB * S_PITCH;
    static constexpr size_t SMEM = size_t(PA * X_PLANE + PB * S_PLANE) * 2;
};

template <class X, int PA, int PB, int NT, bool RANK_ROWS>
__global__ void __launch_bounds__(RANK_THREADS)
    stack_tile_kernel(int C, X x, bool x_wide, const float *S, long long lds, bool scaled, Adapters ad, Groups g,
                      float *partial) {
    using Z = StackTile<X, PA, PB, NT>;
    constexpr int SN = (SLAB * NT + RANK_THREADS - 1) / RANK_THREADS;
    extern __shared__ __align__(16) unsigned char smem_rank[];
    bf16 *xs = reinterpret_cast<bf16 *>(smem_rank), *ss = xs + PA * Z::X_PLANE;
    if (int(blockIdx.y) >= g.totals[1]) return;
    const int4 chunk = g.chunks[blockIdx.y];
    const int a = chunk.x, n = chunk.z, c0 = blockIdx.x * Z::COLS, rank = ad.rank(a);
    const float scale = scaled ? 1.0f : ad.scale(a);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    float xv[4][8], sv[SN][8];
    auto load = [&](int i0) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {   // 64 rows x 16 octets
            const int o = threadIdx.x + h * RANK_THREADS, m = i0 + o / 16, c = c0 + (o % 16) * 8;
            const int i = m < n ? g.perm[chunk.y + m] : -1;
            if (i >= 0 && x_wide && c + 8 <= C) {
                x.at8(i, c, xv[h]);
            } else {
#pragma unroll
                for (int d = 0; d < 8; ++d) xv[h][d] = (i >= 0 && c + d < C) ? x.at(i, c + d) : 0.0f;
            }
        }
#pragma unroll
        for (int h = 0; h < SN; ++h) {   // 64 rows x NT octets
            const int o = threadIdx.x + h * RANK_THREADS, m = i0 + o / NT, r = (o % NT) * 8;
            const bool in = o < SLAB * NT && m < n;
            const long long at = in ? g.perm[chunk.y + m] * lds : 0;
#pragma unroll
            for (int d = 0; d < 8; ++d) sv[h][d] = in && r + d < rank ? S[at + r + d] * scale : 0.0f;
        }
    };

    float sum[NT][4] = {};
    load(0);
    for (int i0 = 0; i0 < n; i0 += SLAB) {
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const int o = threadIdx.x + h * RANK_THREADS;
            stage8<PA>(xs + (o / 16) * Z::X_PITCH + (o % 16) * 8, Z::X_PLANE, xv[h]);
        }
#pragma unroll
        for (int h = 0; h < SN; ++h) {
            const int o = threadIdx.x + h * RANK_THREADS;
            if (o < SLAB * NT) {
                float part[8][3];
#pragma unroll
                for (int d = 0; d < 8; ++d) split_parts(sv[h][d], part[d]);
                bf16 *to = ss + (o / NT) * Z::S_PITCH + (o % NT) * 8;
#pragma unroll
                for (int q = 0; q < PB; ++q)
                    *reinterpret_cast<uint4 *>(to + q * Z::S_PLANE) =
                        make_uint4(pack_bf16(part[0][q], part[1][q]), pack_bf16(part[2][q], part[3][q]),
                                   pack_bf16(part[4][q], part[5][q]), pack_bf16(part[6][q], part[7][q]));
            }
        }
        __syncthreads();
        if (i0 + SLAB < n) load(i0 + SLAB);
        float acc[NT][4] = {};
        auto products = [&](int qa, int qb) {
#pragma unroll
            for (int kk = 0; kk < SLAB; kk += 16) {
                uint32_t fa[4];
                ldmatrix4<true>(fa, shared_address(xs + qa * Z::X_PLANE +
                                                   (kk + (lane & 7) + ((lane >> 4) & 1) * 8) * Z::X_PITCH +
                                                   warp * 16 + ((lane >> 3) & 1) * 8));
#pragma unroll
                for (int t = 0; t < NT; t += 2) {
                    uint32_t fb[4];
                    ldmatrix4<true>(fb, shared_address(ss + qb * Z::S_PLANE + (kk + (lane & 15)) * Z::S_PITCH + t * 8 +
                                                       ((lane >> 4) & 1) * 8));
                    mma16816(acc[t], fa, fb[0], fb[1]);
                    mma16816(acc[t + 1], fa, fb[2], fb[3]);
                }
            }
        };
#pragma unroll
        for (int rest = 2; rest > 0; --rest)
#pragma unroll
            for (int qa = 0; qa <= rest; ++qa)
                if (qa < PA && rest - qa < PB) products(qa, rest - qa);
        products(0, 0);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int d = 0; d < 4; ++d) sum[t][d] += acc[t][d];
    }
    float *out = partial + (long long)blockIdx.y * C * ad.R;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int c = c0 + warp * 16 + (lane >> 2) + (d / 2) * 8, r = t * 8 + (lane & 3) * 2 + (d & 1);
            if (c < C && r < ad.R) out[RANK_ROWS ? (long long)r * C + c : (long long)c * ad.R + r] = sum[t][d];
        }
}

// The chunks' partial sums of an adapter (blockIdx.y) added in order; rows x cols is the
// shape of its gradient (the rank down the rows where RANK_ROWS).
template <class T>
__global__ void __launch_bounds__(256)
    stack_finish_kernel(int rows, int cols, const float *__restrict__ partial, Groups g, Stack<T> out) {
    const int a = blockIdx.y, q0 = g.chunk_begin[a], q1 = g.chunk_begin[a + 1];
    const long long plane = (long long)rows * cols;
    T *to = out.matrix(a);
    for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < plane; t += (long long)gridDim.x * 256) {
        float sum = 0.0f;
#pragma unroll 4
        for (int q = q0; q < q1; ++q) sum += partial[q * plane + t];
        const long long i = t / cols;
        to[i * out.ld + (t - i * cols)] = from_f32<T>(sum);
    }
}

}  // namespace sgl
