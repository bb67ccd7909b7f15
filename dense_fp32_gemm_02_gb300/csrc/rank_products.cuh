// rank_products.cuh -- what the adapter layer computes from the rank side's sums: their
// scaled forms, and the gradients of the stack, X^T * S over the rows of a group (C x R).
//
// The gradients are skinny (at most 128 wide), so they are bound by reading X once, and
// the rows of a group lie anywhere in X.  So the warp-level MMA (m16n8k16, bfloat16, fp32
// accumulators) is fast enough: its operands come from shared memory that asynchronous
// copies fill row by row, from any alignment, several slabs ahead.  A float32 element is
// three bfloat16 parts (see parts_gemm.cuh), which the call has in memory for its product,
// or makes on the way; a checkpoint's is one.
//
// A block only ever holds rows of one adapter: nothing of another one's is multiplied,
// not even by zero.
//
// The MMA's additions truncate, so a slab's products (at most 64 of the contraction) add up from
// zero, the small pairs of parts apart, and then go to fp32 sums, round to nearest:
// four additions of full size to a slab truncate, 5e-7 at most.
#pragma once

#include <type_traits>

#include "lora.cuh"

namespace sgl {

constexpr int SLAB = 64;              // of the contraction
constexpr int RANK_THREADS = 256;

__device__ __forceinline__ uint32_t shared_address(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
template <bool TRANSPOSE>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const bf16 *p) {
    const uint32_t at = shared_address(p);
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

// Two elements as a packed pair of each of three parts.
__device__ __forceinline__ void pair_parts(float x, float y, uint32_t (&part)[3]) {
    float px[3], py[3];
    split_parts(x, px);
    split_parts(y, py);
#pragma unroll
    for (int q = 0; q < 3; ++q) part[q] = pack_exact(px[q], py[q]);
}

// 16 bytes of shared memory from `n` elements at p (the rest zero): an asynchronous copy
// where p is 16-byte aligned, four of them for float32, else (bfloat16) loads and a store.
template <class T>
__device__ __forceinline__ void fill16(T *to, const T *p, int n, bool wide) {
    constexpr int PER = 16 / int(sizeof(T));
    n = max(0, min(PER, n));
    if (wide) {
        sg::cp_async16(shared_address(to), p, uint32_t(n) * sizeof(T));
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int d = 0; d < PER; ++d) sg::cp_async4(shared_address(to + d), d < n ? p + d : p, d < n ? 4u : 0u);
    } else {
        alignas(16) T x[PER];
#pragma unroll
        for (int d = 0; d < PER; ++d) x[d] = d < n ? p[d] : T(0.0f);
        *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(x);
    }
}

// ------------------------------------------------------------------ rank side
// What the rank side leaves behind: S (M x R, scaled), unscaled for the caller in H, and
// S's parts in the planes of Groups and, for the stack's gradients, as rows of `pitch` columns, zero
// past the rank: `s_rows` of S and `h_rows` of the scaled H that the caller gave.  What is
// null is left out.  `filled`: those rows meet matrices of one part, whose infinities meet all
// parts of a sum.
struct RankSide {
    float *S, *H;
    long long ldh;
    bf16 *planes, *s_rows, *h_rows;
    int pitch;
    bool filled;
};

// The parts of x with none of them zero: the least normal number, of x's sign, in the place of a
// zero (under 2^-30 of x; a smaller x keeps its zeros), because infinity times zero is NaN.
__device__ __forceinline__ void fill_parts(float x, float (&part)[3]) {
    const float least = fabsf(x) >= 0x1p-96f ? copysignf(0x1p-126f, x) : 0.0f;
    part[1] = part[1] == 0.0f ? least : part[1];
    part[2] = part[2] == 0.0f ? least : part[2];
}

// The ranges' partial sums of the rank side added in order, WARPS warps to a row.  A row
// whose adapter holds something that is not finite keeps the product from its tile's planes.
template <int WARPS>
__global__ void __launch_bounds__(256)
    rank_finish_kernel(int M, int ranges, const float *__restrict__ partial, long long partial_plane, Adapters ad,
                       Groups g, RankSide to) {
    constexpr int ROWS = 8 / WARPS, THREADS = 32 * WARPS;
    __shared__ float own_s[ROWS][128], own_h[ROWS][128];
    const int t = threadIdx.x % THREADS, lane = t & 31, warp = t >> 5, in_block = threadIdx.x / THREADS;
    const long long row = (long long)blockIdx.x * ROWS + in_block, i = row < M ? row : M - 1;
    const int a = ad.of_row(i), rank = a < 0 ? 0 : ad.rank(a);
    const float scale = a < 0 ? 0.0f : ad.scale(a);
    float *S = own_s[in_block], *H = own_h[in_block];
    sg::wait_prerequisites();
    sg::launch_dependents();
    const int4 planes = to.planes ? g.planes[i / 256] : make_int4(0, 0, 0, 0);
    const int first = to.planes ? g.position[i] * g.width : 0;
    const bool unclean = to.planes && rank > 0 && g.unclean[a];
    const bool fits = SG_IN_RANGE(ad.R <= g.width && ad.R <= 128 && first >= 0 &&
                                  (!to.planes || rank == 0 || first + g.width <= 64 * planes.y) &&
                                  (!planes.z || (planes.x >= 0 && planes.x + planes.y <= g.capacity)));
    for (int r = t; r < ad.R; r += THREADS) {
        float sum = 0.0f, h = 0.0f;
        if (r < rank) {
            if (to.h_rows) h = to.H[i * to.ldh + r];
#pragma unroll 8
            for (int s = 0; s < ranges; ++s) sum += partial[s * partial_plane + i * g.width + r];
        }
        const float scaled = r < rank ? sum * scale : 0.0f;
        S[r] = scaled;
        H[r] = r < rank ? h * scale : 0.0f;
        if (row < M) {
            to.S[i * ad.R + r] = scaled;
            if (to.H && !to.h_rows) to.H[i * to.ldh + r] = sum;
        }
    }
    __syncthreads();
    if (row >= M || !fits) return;
    auto rows_of = [&](bf16 *rows, const float *x) {   // a row as parts
        for (int r = 2 * t; r < to.pitch; r += 2 * THREADS) {
            const float xr = r < rank ? x[r] : 0.0f, yr = r + 1 < rank ? x[r + 1] : 0.0f;
            float px[3], py[3];
            split_parts(xr, px);
            split_parts(yr, py);
            if (to.filled) fill_parts(xr, px), fill_parts(yr, py);
#pragma unroll
            for (int q = 0; q < S_PARTS; ++q)
                *reinterpret_cast<uint32_t *>(rows + ((long long)q * M + i) * to.pitch + r) = pack_exact(px[q], py[q]);
        }
    };
    if (to.h_rows) rows_of(to.h_rows, H);
    if (to.s_rows) rows_of(to.s_rows, S);
    if (unclean && t == 0) atomicExch(&g.planes[i / 256].z, 0);
    if (!planes.z) return;
    for (int s = warp; s < planes.y; s += WARPS) {
        const int r = s * 64 + 2 * lane - first;
        const float x = r >= 0 && r < rank ? S[r] : 0.0f;
        const float y = r + 1 >= 0 && r + 1 < rank ? S[r + 1] : 0.0f;
        uint32_t part[3];
        pair_parts(x, y, part);
#pragma unroll
        for (int q = 0; q < S_PARTS; ++q)
            *reinterpret_cast<uint32_t *>(
                to.planes + (((long long)q * g.capacity + planes.x + s) * 256 + i % 256) * 64 + 2 * lane) = part[q];
    }
}

// ------------------------------------------------------------------ stack gradients
// X^T * S over a chunk of rows of a group, 128 columns of X: 8 warps, 16 columns x the
// whole rank each.  partial[chunk] is C x R, or R x C where RANK_ROWS.
template <class X>
struct ElementOf;
template <class T>
struct ElementOf<Rows<T>> {
    using type = T;
    static constexpr int PARTS = sizeof(T) == 4 ? 3 : 1;
};
template <>
struct ElementOf<Act8Rows> {
    using type = signed char;
    static constexpr int PARTS = 1;
};
// A float32 matrix whose parts are there already, `plane` apart, 16-byte aligned rows.
struct PartRows {
    const bf16 *p;
    long long ld, plane;
};
template <>
struct ElementOf<PartRows> {
    using type = bf16;
    static constexpr int PARTS = 3;
};

template <class X, int NT>
struct StackTile {
    using E = typename ElementOf<X>::type;
    static constexpr int PA = ElementOf<X>::PARTS, PB = S_PARTS, COLS = 128;
    // float32: rows 4 banks apart; bfloat16 and q: 16 bytes past a multiple of 128
    static constexpr int X_PITCH = COLS + (sizeof(E) == 4 ? 4 : 16 / int(sizeof(E)));
    static constexpr int X_PLANES = sizeof(E) == 2 ? PA : 1, S_PITCH = NT * 8 + 8;
    static constexpr int ROW_BYTES = X_PLANES * X_PITCH * int(sizeof(E)) + PB * S_PITCH * 2 + (sizeof(E) == 1 ? 4 : 0);
    // Rows to a slab, and slabs in the ring: several blocks to an SM hide more than a
    // deeper ring does (4096 x 4096 bfloat16, rank 32, two parts of S: 28 us with two of 4
    // slabs, 22 with four of 2).
    static constexpr int DEPTH = SLAB * ROW_BYTES <= 56 * 1024 ? SLAB : SLAB / 2;
    static constexpr int X_PLANE = DEPTH * X_PITCH, X_BYTES = X_PLANES * X_PLANE * int(sizeof(E));
    static constexpr int S_PLANE = DEPTH * S_PITCH, S_BYTES = PB * S_PLANE * 2;
    static constexpr int E_BYTES = sizeof(E) == 1 ? DEPTH * 4 : 0;   // a row's four exponents
    static constexpr int STAGE = X_BYTES + S_BYTES + E_BYTES;
    static constexpr int STAGES = 3 * STAGE <= 74 * 1024 ? 3 : 2;
    static constexpr size_t SMEM = size_t(STAGES) * STAGE;
};
constexpr int CHUNK_ROWS = 512;   // of a chunk at most

template <class X>
struct StackWork {
    int C;
    X x;
    bool wide;
    const bf16 *s;   // parts of S: PB x M rows of `pitch` columns
    float *partial;
};

template <class X, int NT, bool RANK_ROWS>
__device__ __forceinline__ void stack_tile(const StackWork<X> &w, int bx, int by, int M, int pitch, const Adapters &ad,
                                           const Groups &g, unsigned char *smem, int *rows) {
    using Z = StackTile<X, NT>;
    using E = typename Z::E;
    constexpr int PA = Z::PA, PB = Z::PB, PER = 16 / int(sizeof(E)), STAGES = Z::STAGES, DEPTH = Z::DEPTH;
    const int4 chunk = g.chunks[by];
    const int n = chunk.z, c0 = bx * Z::COLS, C = w.C;
    if (n == 0) return;
    const X &x = w.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (!SG_IN_RANGE(by < g.max_chunks && n > 0 && n <= CHUNK_ROWS && chunk.y >= 0 && (long long)chunk.y + n <= M)) return;
    for (int m = threadIdx.x; m < n; m += RANK_THREADS) {
        const int row = g.perm[chunk.y + m];
        rows[m] = SG_IN_RANGE(row >= 0 && row < M) ? row : 0;
    }
    __syncthreads();

    auto fill = [&](int stage, int i0) {
        E *xs = reinterpret_cast<E *>(smem + stage * Z::STAGE);
        bf16 *ss = reinterpret_cast<bf16 *>(smem + stage * Z::STAGE + Z::X_BYTES);
#pragma unroll
        for (int o = threadIdx.x; o < DEPTH * Z::COLS / PER; o += RANK_THREADS) {
            const int m = o / (Z::COLS / PER), c = (o % (Z::COLS / PER)) * PER;
            const bool in = i0 + m < n && c0 + c < C && SG_IN_RANGE(m < DEPTH && c + PER <= Z::X_PITCH);
            const long long i = in ? rows[i0 + m] : 0;
            if constexpr (sizeof(E) == 1) {
                E *to = xs + m * Z::X_PITCH + c;
                const E *p = x.q + i * x.ldq + c0 + c;
                const int count = in ? min(PER, C - c0 - c) : 0;
                if (w.wide) {
                    sg::cp_async16(shared_address(to), in ? p : x.q, uint32_t(count));
                } else {
                    alignas(16) E b[PER];
#pragma unroll
                    for (int d = 0; d < PER; ++d) b[d] = d < count ? p[d] : E(0);
                    *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(b);
                }
            } else if constexpr (std::is_same<X, PartRows>::value) {
#pragma unroll
                for (int q = 0; q < 3; ++q)
                    fill16(xs + q * Z::X_PLANE + m * Z::X_PITCH + c, in ? x.p + q * x.plane + i * x.ld + c0 + c : x.p,
                           in ? C - c0 - c : 0, true);
            } else {
                fill16(xs + m * Z::X_PITCH + c, in ? x.p + i * x.ld + c0 + c : x.p, in ? C - c0 - c : 0, w.wide);
            }
        }
#pragma unroll
        for (int q = 0; q < PB; ++q)
#pragma unroll
            for (int o = threadIdx.x; o < DEPTH * NT; o += RANK_THREADS) {
                const int m = o / NT, r = (o % NT) * 8;
                const bool in = i0 + m < n && SG_IN_RANGE(m < DEPTH && r + 8 <= Z::S_PITCH && r + 8 <= pitch);
                const long long i = in ? rows[i0 + m] : 0;
                sg::cp_async16(shared_address(ss + q * Z::S_PLANE + m * Z::S_PITCH + r),
                               w.s + ((long long)q * M + i) * pitch + r, in ? 16u : 0u);
            }
        if constexpr (sizeof(E) == 1) {
            signed char *es = reinterpret_cast<signed char *>(ss) + Z::S_BYTES;
            const int m = threadIdx.x / 4, block = c0 / ACT8_BLOCK + threadIdx.x % 4;
            const bool in = i0 + m < n && block * ACT8_BLOCK < C;
            if (m < DEPTH) es[threadIdx.x] = in ? x.e[rows[i0 + m] * x.lde + block] : E(0);
        }
    };

    float sum[NT][4] = {};
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
        if (s * DEPTH < n) fill(s, s * DEPTH);
        sg::cp_async_commit();
    }
    int stage = 0;
    for (int i0 = 0; i0 < n; i0 += DEPTH) {
        sg::cp_async_wait<STAGES - 2>();
        __syncthreads();   // this slab has landed, and the stage filled next has been read
        if (i0 + (STAGES - 1) * DEPTH < n) fill((stage + STAGES - 1) % STAGES, i0 + (STAGES - 1) * DEPTH);
        sg::cp_async_commit();
        const E *xs = reinterpret_cast<const E *>(smem + stage * Z::STAGE);
        const bf16 *ss = reinterpret_cast<const bf16 *>(smem + stage * Z::STAGE + Z::X_BYTES);
        const signed char *es = reinterpret_cast<const signed char *>(ss) + Z::S_BYTES;
        float acc[NT][4] = {};
        // the columns' fragment of part qa at rows kk .. kk + 15: element (column, row)
        auto columns = [&](uint32_t (&fa)[PA][4], int kk) {
            if constexpr (sizeof(E) == 2) {
#pragma unroll
                for (int q = 0; q < PA; ++q)
                    ldmatrix4<true>(fa[q], reinterpret_cast<const bf16 *>(xs) + q * Z::X_PLANE +
                                               (kk + (lane & 7) + ((lane >> 4) & 1) * 8) * Z::X_PITCH + warp * 16 +
                                               ((lane >> 3) & 1) * 8);
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const int k = kk + (lane & 3) * 2 + (d >> 1) * 8, c = warp * 16 + (lane >> 2) + (d & 1) * 8;
                    if constexpr (sizeof(E) == 4) {
                        uint32_t part[3];
                        pair_parts(xs[k * Z::X_PITCH + c], xs[(k + 1) * Z::X_PITCH + c], part);
                        fa[0][d] = part[0], fa[1][d] = part[1], fa[2][d] = part[2];
                    } else {
                        const signed char *e = es + k * 4 + warp / 2;
                        fa[0][d] = pack_bf16(float(xs[k * Z::X_PITCH + c]) * act8_step(e[0]),
                                             float(xs[(k + 1) * Z::X_PITCH + c]) * act8_step(e[4]));
                    }
                }
            }
        };
        // The small pairs of parts have sums of their own; at the widest rank, for which that
        // takes too many registers, they come first instead, in a pass of their own.
        constexpr bool APART = NT <= 8;
        float small[APART ? NT : 1][4] = {};
#pragma unroll
        for (int pass = APART ? 1 : 0; pass < 2; ++pass) {
#pragma unroll
            for (int kk = 0; kk < DEPTH; kk += 16) {
                uint32_t fa[PA][4];
                columns(fa, kk);
#pragma unroll
                for (int qb = APART || pass == 0 ? PB - 1 : 0; qb >= 0; --qb)
#pragma unroll
                    for (int t = 0; t < NT; t += 2) {
                        uint32_t fb[4];
                        ldmatrix4<true>(fb, ss + qb * Z::S_PLANE + (kk + (lane & 15)) * Z::S_PITCH + t * 8 +
                                                ((lane >> 4) & 1) * 8);
#pragma unroll
                        for (int qa = PA - 1; qa >= 0; --qa) {
                            const bool minor = qa + qb > 0;
                            if (qa + qb > 2 || (!APART && minor != (pass == 0))) continue;
                            mma16816(APART && minor ? small[APART ? t : 0] : acc[t], fa[qa], fb[0], fb[1]);
                            mma16816(APART && minor ? small[APART ? t + 1 : 0] : acc[t + 1], fa[qa], fb[2], fb[3]);
                        }
                    }
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int d = 0; d < 4; ++d) sum[t][d] += APART ? acc[t][d] + small[APART ? t : 0][d] : acc[t][d];
        stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    float *out = w.partial + (long long)by * C * ad.R;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int c = c0 + warp * 16 + (lane >> 2) + (d / 2) * 8, r = t * 8 + (lane & 3) * 2 + (d & 1);
            if (c < C && r < ad.R) out[RANK_ROWS ? (long long)r * C + c : (long long)c * ad.R + r] = sum[t][d];
        }
}

// Blocks to an SM that the registers are limited for.  (float32 of rank 64, 4483 x 5120 x
// 5760: 158 us at one, 125 at two.)
constexpr int stack_blocks(int parts, int nt) { return nt <= 4 ? (parts == 1 ? 4 : 2) : nt == 8 ? 2 : 1; }

// Both gradients: X^T G (C = K columns of X, 128 to a block) and H^T dY (N columns of dY),
// each for max_chunks chunks.
template <class XA, class XB, int NT>
__global__ void __launch_bounds__(RANK_THREADS, stack_blocks(ElementOf<XB>::PARTS, NT))
    stack_tile_kernel(StackWork<XA> wa, StackWork<XB> wb, int M, int pitch, Adapters ad, Groups g) {
    extern __shared__ __align__(16) unsigned char smem_stack[];
    __shared__ int rows[CHUNK_ROWS];
    sg::wait_prerequisites();
    sg::launch_dependents();
    const int across = (wa.C + 127) / 128 + (wb.C + 127) / 128, bx = blockIdx.x % across, by = blockIdx.x / across;
    if (bx < (wa.C + 127) / 128)
        stack_tile<XA, NT, false>(wa, bx, by, M, pitch, ad, g, smem_stack, rows);
    else
        stack_tile<XB, NT, true>(wb, bx - (wa.C + 127) / 128, by, M, pitch, ad, g, smem_stack, rows);
}

// The chunks' partial sums of an adapter (blockIdx.y) added in order: K x R to dA, then
// R x N to dB.  Past the adapter's rank there is zero: the partial sums hold products of S's zeros
// there, which are NaN where a row of X or dY holds an infinity or a NaN.
template <class T>
__global__ void __launch_bounds__(256)
    stack_finish_kernel(int K, int N, Adapters ad, const float *__restrict__ pa, const float *__restrict__ pb, Groups g,
                        Stack<T> dA, Stack<T> dB) {
    sg::wait_prerequisites();
    sg::launch_dependents();
    const int a = blockIdx.y, R = ad.R, rank = ad.rank(a), q0 = g.chunk_begin[a], q1 = g.chunk_begin[a + 1];
    if (!SG_IN_RANGE(a < ad.L && q0 >= 0 && q0 <= q1 && q1 <= g.max_chunks)) return;
    const long long plane_a = (long long)K * R, plane_b = (long long)R * N;
    for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < plane_a + plane_b;
         t += (long long)gridDim.x * 256) {
        const bool first = t < plane_a;
        const long long u = first ? t : t - plane_a, plane = first ? plane_a : plane_b;
        const float *p = (first ? pa : pb) + u;
        const int cols = first ? R : N;
        const long long i = u / cols;
        const int r = int(first ? u - i * cols : i);
        float sum = 0.0f;
#pragma unroll 4
        for (int q = q0; q < (r < rank ? q1 : q0); ++q) sum += p[q * plane];
        const Stack<T> &out = first ? dA : dB;
        if (SG_IN_RANGE(i >= 0 && i < (first ? K : R) && r >= 0 && r < R)) out.matrix(a)[i * out.ld + (u - i * cols)] = from_f32<T>(sum);
    }
}

}  // namespace sgl
