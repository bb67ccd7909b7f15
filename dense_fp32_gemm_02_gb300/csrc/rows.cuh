// rows.cuh -- the adapter layer for few rows (a decode step): Y = X W + bias + rank side.
//
// Bound by reading W once (and of the stack what the rows use).  The contraction is
// split over the grid, each range's sums go to memory, and a last kernel adds the ranges
// in order and applies the rest.  The product itself, by the count of rows:
//   up to 8             stream_rows_kernel: W to registers 16 bytes at a time, fp32 FMAs
//                       (bfloat16 of 3 and more rows: unless W is large);
//   float32 up to 64    few_rows_kernel: W through shared memory, the warp-level MMA on
//                       three bfloat16 parts, split in registers;
//   else                parts_gemm.cuh.
// At 4096 x 4096 without adapters, us: bfloat16 (W is 5.0 of them) 1 row 9.6, 4 rows 12.5,
// and by parts_gemm 8 rows 15 (by FMAs 20.5, 16 rows 34), 64 rows 17.6 (the
// warp-level MMA took 32: its operands pass through shared memory five times); float32 (W
// 9.9) 1 row 14.3, 8 rows 21.3, 16 rows 22.5 (by FMAs 43), 64 rows 50.  At 1024 x 1024 8 rows of
// bfloat16 take 5.7 by FMAs, 9 rows 8.4 by parts_gemm: hence 8 for both.
// The rank side is taken row by row, each with its own adapter, by blocks of their own:
// in the product's launch where all blocks fit the GPU at once, else in one just after,
// which runs beside it where it leaves room (64 x 4096 x 4096 bfloat16 with rank 16: 22 us;
// before it 23.6, because the product's blocks then wait for shared memory).
#pragma once

#include <algorithm>

#include "rank_products.cuh"

namespace sgl {

constexpr int FEW_ROWS = 1280, STREAM_ROWS = 8, MMA_ROWS = 64, ROWS_COLS = 128;

// The work: `across` x `ranges` blocks of the product, then M x `rank_ranges` blocks of
// the rank side.
struct RowsWork {
    int M, N, K;
    int across, ranges, range;
    int rank_ranges, rank_range;
    bool x_wide, v_wide;
    float *partial;        // ranges x M x N
    float *rank_partial;   // rank_ranges x M x R
};

// The split of K over the grid: the count of ranges (whole `step`s, none above `longest`)
// whose waves of blocks take the fewest steps, with two for filling and emptying; partial
// sums (8 bytes of traffic per row and column) of at most half of what W takes.  `matrices` like W
// are multiplied together.
inline void split_rows(RowsWork &w, int cols, int step, int longest, long long slots, size_t element, int matrices = 1) {
    w.across = (w.N + cols - 1) / cols;
    const long long steps = (w.K + step - 1LL) / step;
    const long long fewest = (w.K + (long long)longest - 1) / longest;
    const long long most = std::max(fewest, std::min(steps, (long long)w.K * (long long)element / (16LL * w.M)));
    long long least = 0;
    for (long long n = fewest; n <= std::min(most, fewest + 64); ++n) {
        const long long per = (steps + n - 1) / n;
        const long long cost = ((matrices * w.across * n + slots - 1) / slots) * (per + 2);
        if (n == fewest || cost < least) least = cost, w.range = int(per * step);
    }
    w.ranges = int((w.K + (long long)w.range - 1) / w.range);
}

// The rank side of one row over one range.  Lanes along the rank, 16 bytes each, and in
// groups along the range; a thread's sums, then its warp's groups, then the warps.
template <class T>
__device__ __forceinline__ void rank_of_row(const RowsWork &w, int b, const Rows<T> &X, const Stack<const T> &V,
                                            const Adapters &ad, float *sums) {
    constexpr int PER = 16 / int(sizeof(T));
    const int i = b / w.rank_ranges, q = b - i * w.rank_ranges;
    const int a = ad.of_row(i);
    const int rank = a < 0 ? 0 : ad.rank(a);
    if (rank == 0) return;   // nothing reads this row's sums
    if (!SG_IN_RANGE(b >= 0 && i < w.M && q >= 0 && q < w.rank_ranges && ad.R <= 128)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int along = 1;           // lanes along the rank: a power of two, up to 16 (32 for float32)
    while (along * PER < ad.R) along *= 2;
    const int groups = RANK_THREADS / along, r0 = (threadIdx.x & (along - 1)) * PER, group = threadIdx.x / along;
    const int c0 = q * w.rank_range, c1 = min(w.K, c0 + w.rank_range);
    const T *x = X.p + i * X.ld, *v = V.matrix(a) + r0;
    float sum[PER] = {};
    if (r0 < rank) {
        if (w.v_wide && r0 + PER <= ad.R) {
#pragma unroll 4
            for (int c = c0 + group; c < c1; c += groups) {
                const float xc = to_f32(x[c]);
                float y[PER];
                if constexpr (PER == 8) load8(v + c * V.ld, y); else load4(v + c * V.ld, y);
#pragma unroll
                for (int d = 0; d < PER; ++d) sum[d] = fmaf(xc, r0 + d < rank ? y[d] : 0.0f, sum[d]);
            }
        } else {
#pragma unroll 2
            for (int c = c0 + group; c < c1; c += groups) {
                const float xc = to_f32(x[c]);
#pragma unroll
                for (int d = 0; d < PER; ++d) sum[d] = fmaf(xc, r0 + d < rank ? to_f32(v[c * V.ld + d]) : 0.0f, sum[d]);
            }
        }
    }
#pragma unroll
    for (int d = 0; d < PER; ++d)
        for (int o = 16; o >= along; o >>= 1) sum[d] += __shfl_xor_sync(0xffffffffu, sum[d], o);
    if (lane < along && SG_IN_RANGE(r0 + PER <= 128)) {
#pragma unroll
        for (int d = 0; d < PER; ++d) sums[warp * 128 + r0 + d] = sum[d];
    }
    __syncthreads();
    const int r = threadIdx.x;
    if (r < rank) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < RANK_THREADS / 32; ++k) s += sums[k * 128 + r];
        w.rank_partial[((long long)q * w.M + i) * ad.R + r] = s;
    }
}
constexpr int RANK_SUMS = RANK_THREADS / 32 * 128;

template <class T>
__global__ void __launch_bounds__(RANK_THREADS)
    few_rows_rank_kernel(RowsWork w, Rows<T> X, Stack<const T> V, Adapters ad) {
    __shared__ float sums[RANK_SUMS];
    sg::launch_dependents();
    rank_of_row(w, int(blockIdx.x), X, V, ad, sums);   // (inputs, and workspace of its own: host_state.h)
    if (blockIdx.x == 0) sg::wait_prerequisites();   // this kernel's end is also that of the product's
}

// ------------------------------------------------------------------ up to 8 rows
// A block to 32 x 16 bytes of columns and a range of at most STREAM_RANGE of K: its warps
// take 8 rows of W at a time, all loads before the first use.  X's range stands in shared
// memory as fp32, MR rows next to each other.  WIDE: 16-byte loads, a lane's columns
// together; else single elements, 32 lanes next to each other.
constexpr int STREAM_RANGE = 512, STREAM_DEPTH = 8;

constexpr int stream_blocks(int rows) { return rows <= 4 ? 3 : 2; }   // to an SM

template <class T, int MR>
struct StreamRows {
    static constexpr int COLS = 32 * 16 / int(sizeof(T)), WARPS = RANK_THREADS / 32;
    static constexpr int XS = STREAM_RANGE * MR, RED = WARPS * COLS * (MR < 4 ? MR : 4);
    static constexpr int FLOATS = XS > RED ? (XS > RANK_SUMS ? XS : RANK_SUMS) : (RED > RANK_SUMS ? RED : RANK_SUMS);
};

// Block `block` of the product; its sums go to partial[range][row][column].
template <class T, int MR, bool WIDE>
__device__ __forceinline__ void stream_rows(const RowsWork &w, int block, const Rows<T> &X, const T *W, long long ldw,
                                            float *partial, float *sm) {
    constexpr int PER = 16 / int(sizeof(T)), COLS = StreamRows<T, MR>::COLS, WARPS = StreamRows<T, MR>::WARPS;
    [[maybe_unused]] constexpr int RED = StreamRows<T, MR>::RED;
    const int n0 = (block % w.across) * COLS, q = block / w.across;
    const int k0 = q * w.range, kn = min(w.range, w.K - k0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (!SG_IN_RANGE(kn > 0 && kn <= STREAM_RANGE && k0 + kn <= w.K && n0 < w.N && q < w.ranges && w.M <= MR)) return;
    auto column = [&](int e) { return n0 + (WIDE ? lane * PER + e : e * 32 + lane); };
    auto load = [&](int k) {   // 16 bytes of row k0 + k of W, zero past its end
        const T *p = W + (k0 + k) * ldw;
        if (WIDE && column(PER - 1) < w.N) return *reinterpret_cast<const uint4 *>(p + column(0));
        alignas(16) T v[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) v[e] = column(e) < w.N ? p[column(e)] : T(0.0f);
        return *reinterpret_cast<const uint4 *>(v);
    };
    for (int t = threadIdx.x; t < kn * MR; t += RANK_THREADS) {
        const int m = t / kn, k = t - m * kn;
        sm[k * MR + m] = m < w.M ? X.at(m, k0 + k) : 0.0f;
    }
    __syncthreads();
    float2 acc[MR][PER / 2] = {};
    for (int k = warp * STREAM_DEPTH; k < kn; k += WARPS * STREAM_DEPTH) {
        uint4 v[STREAM_DEPTH];
#pragma unroll
        for (int u = 0; u < STREAM_DEPTH; ++u) v[u] = k + u < kn ? load(k + u) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < STREAM_DEPTH; ++u) {
            const float *x = sm + min(k + u, kn - 1) * MR;
            const bool in = k + u < kn;   // (a row past the range is 0 * x: x may be NaN)
            float2 y[PER / 2];
            if constexpr (PER == 8) {
                y[0] = make_float2(bf16_lo(v[u].x), bf16_hi(v[u].x)), y[1] = make_float2(bf16_lo(v[u].y), bf16_hi(v[u].y));
                y[2] = make_float2(bf16_lo(v[u].z), bf16_hi(v[u].z)), y[3] = make_float2(bf16_lo(v[u].w), bf16_hi(v[u].w));
            } else {
                y[0] = make_float2(__uint_as_float(v[u].x), __uint_as_float(v[u].y));
                y[1] = make_float2(__uint_as_float(v[u].z), __uint_as_float(v[u].w));
            }
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                const float xm = in ? x[m] : 0.0f;
#pragma unroll
                for (int e = 0; e < PER / 2; ++e) acc[m][e] = sg::ffma2(make_float2(xm, xm), y[e], acc[m][e]);
            }
        }
    }
    float *out = partial + (long long)q * w.M * w.N;
#pragma unroll
    for (int m0 = 0; m0 < MR; m0 += 4) {
        __syncthreads();
#pragma unroll
        for (int m = m0; m < m0 + 4 && m < MR; ++m)
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const float s = e & 1 ? acc[m][e / 2].y : acc[m][e / 2].x;
                sm[((m - m0) * WARPS + warp) * COLS + (WIDE ? lane * PER + e : e * 32 + lane)] = s;
            }
        __syncthreads();
        for (int t = threadIdx.x; t < min(4, MR) * COLS; t += RANK_THREADS) {
            const int m = m0 + t / COLS, c = t % COLS;
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < WARPS; ++k) s += sm[((m - m0) * WARPS + k) * COLS + c];
            if (m < w.M && n0 + c < w.N && SG_IN_RANGE(((m - m0 + 1) * WARPS - 1) * COLS + c < RED)) out[(long long)m * w.N + n0 + c] = s;
        }
    }
}

template <class T, int MR, bool WIDE>
__global__ void __launch_bounds__(RANK_THREADS, stream_blocks(MR))
    stream_rows_kernel(RowsWork w, Rows<T> X, const T *W, long long ldw, Stack<const T> V, Adapters ad) {
    __shared__ __align__(16) float sm[StreamRows<T, MR>::FLOATS];
    sg::launch_dependents();
    if (int(blockIdx.x) >= w.across * w.ranges) {
        rank_of_row(w, int(blockIdx.x) - w.across * w.ranges, X, V, ad, sm);
        return;
    }
    stream_rows<T, MR, WIDE>(w, int(blockIdx.x), X, W, ldw, w.partial, sm);
}

// ------------------------------------------------------------------ float32, up to 64 rows
// The warp-level MMA on three bfloat16 parts of each side, six products (parts_gemm.cuh), each
// 16 k from zero, small products first, and then into fp32 sums.  The warps take 32 columns
// each, four apart in a tile, so that a lane reads its columns of four tiles at once, and a
// piece of a slab's k.
//
// Bound by the latency of a slab's steps at 16 rows (4096 x 4096: 22.5 us, W's bytes 9.9; three
// stages of W, or sixteen warps to a block, took 23 and 26) and by the MMAs at 64 (1024
// products per clock and SM: 21 us of 50).  Two TF32 parts, three products at a quarter of
// the rate, took 22 and 60.
template <int MT>
struct FewRows {
    static constexpr int STAGES = 2;   // and two blocks to an SM
    static constexpr int W_PITCH = ROWS_COLS + 4, W_ELEMS = SLAB * W_PITCH;
    static constexpr int X_ROWS = MT * 16, X_PITCH = SLAB + 8, X_PLANE = X_ROWS * X_PITCH;
    static constexpr size_t SMEM = size_t(STAGES) * W_ELEMS * 4 + size_t(X_ROWS) * SLAB * 4 + size_t(3) * X_PLANE * 2;
};

// Four pairs (x[i], y[i]) as packed parts.  Remainders of what is finite need no check.
__device__ __forceinline__ void parts_of_pairs(const float (&x)[4], const float (&y)[4], uint32_t (&part)[3][4]) {
    auto head = [](float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); };
    const float2 one = make_float2(1.0f, 1.0f), minus = make_float2(-1.0f, -1.0f);
    float2 rest[4], all = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        rest[i] = sg::ffma2(make_float2(head(x[i]), head(y[i])), minus, make_float2(x[i], y[i]));
        all = sg::ffma2(rest[i], one, all);
    }
    if (all.x + all.y != all.x + all.y) {   // an infinity or a NaN among them
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t p[3];
            pair_parts(x[i], y[i], p);
            part[0][i] = p[0], part[1][i] = p[1], part[2][i] = p[2];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 s = sg::ffma2(make_float2(head(rest[i].x), head(rest[i].y)), minus, rest[i]);
        part[0][i] = pack_exact(x[i], y[i]);
        part[1][i] = pack_exact(rest[i].x, rest[i].y);
        part[2][i] = pack_exact(s.x, s.y);
    }
}

// d = a * b
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// Block `block` of the product, its sums to partial[range][row][column]; `smem` FewRows<MT>::SMEM bytes.
template <int MT>
__device__ __forceinline__ void few_rows(const RowsWork &w, int block, const Rows<float> &X, const float *W, long long ldw,
                                         bool w_wide, float *partial, unsigned char *smem) {
    using Z = FewRows<MT>;
    constexpr int STAGES = Z::STAGES, WARPS = RANK_THREADS / 32, PIECES = WARPS / 4;   // of a slab's k
    float *ring = reinterpret_cast<float *>(smem);
    float *raw = ring + STAGES * Z::W_ELEMS;                      // X's next slab
    bf16 *xs = reinterpret_cast<bf16 *>(raw + Z::X_ROWS * SLAB);   // this one's parts
    const int n0 = (block % w.across) * ROWS_COLS, q = block / w.across;
    const int k_begin = q * w.range, k_end = min(w.K, k_begin + w.range);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp & 3, piece = warp >> 2;
    if (!SG_IN_RANGE(k_begin < k_end && n0 < w.N && q < w.ranges && w.M <= Z::X_ROWS)) return;

    // every WARPS'th row of the slab to a warp, 16 bytes to a lane or single elements
    auto fill = [&](int stage, int k0) {
        float *to = ring + stage * Z::W_ELEMS + warp * Z::W_PITCH;
        const float *from = W + (k0 + warp) * ldw + n0;
        if (w_wide && n0 + ROWS_COLS <= w.N) {
#pragma unroll
            for (int i = 0; i < SLAB / WARPS; ++i, from += WARPS * ldw) {
                const bool in = k0 + warp + WARPS * i < k_end;
                sg::cp_async16(shared_address(to + i * WARPS * Z::W_PITCH + lane * 4), in ? from + lane * 4 : W, in ? 16u : 0u);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < SLAB / WARPS; ++i, from += WARPS * ldw, to += WARPS * Z::W_PITCH)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int c = lane + 32 * d;
                const bool in = k0 + warp + WARPS * i < k_end && n0 + c < w.N;
                sg::cp_async4(shared_address(to + c), in ? from + c : W, in ? 4u : 0u);
            }
    };
    constexpr int QUADS = Z::X_ROWS * SLAB / 4;   // of a slab of X
    auto fill_x = [&](int k0) {
        if (w.x_wide && k0 + SLAB <= k_end) {
#pragma unroll
            for (int o = threadIdx.x; o < QUADS; o += RANK_THREADS) {
                const int m = o / 16;
                sg::cp_async16(shared_address(raw + o * 4), m < w.M ? X.p + m * X.ld + k0 + (o % 16) * 4 : X.p,
                               m < w.M ? 16u : 0u);
            }
            return;
        }
#pragma unroll
        for (int o = threadIdx.x; o < QUADS * 4; o += RANK_THREADS) {
            const int m = o / SLAB, k = k0 + o % SLAB;
            const bool in = m < w.M && k < k_end;
            sg::cp_async4(shared_address(raw + o), in ? X.p + m * X.ld + k : X.p, in ? 4u : 0u);
        }
    };

    float sum[MT][4][4] = {};   // [16 rows][tile: column 4 c + tile of the warp's 32][fragment]
    fill(0, k_begin);
    fill_x(k_begin);
    sg::cp_async_commit();
    int stage = 0;
    for (int k0 = k_begin; k0 < k_end; k0 += SLAB) {
        sg::cp_async_wait<0>();
        __syncthreads();   // this slab has landed, and the last one has been read
        if (k0 + SLAB < k_end) fill(stage ^ 1, k0 + SLAB);
        for (int o = threadIdx.x; o < QUADS / 2; o += RANK_THREADS) {   // eight elements of a row of X
            float v[4], t[4];
            load4(raw + o * 8, v);
            load4(raw + o * 8 + 4, t);
            uint32_t part[3][4];
            const float x[4] = {v[0], v[2], t[0], t[2]}, y[4] = {v[1], v[3], t[1], t[3]};
            parts_of_pairs(x, y, part);
#pragma unroll
            for (int p = 0; p < 3; ++p)
                *reinterpret_cast<uint4 *>(xs + p * Z::X_PLANE + (o / 8) * Z::X_PITCH + (o % 8) * 8) =
                    make_uint4(part[p][0], part[p][1], part[p][2], part[p][3]);
        }
        __syncthreads();   // X's parts are there, and its slab has been read
        if (k0 + SLAB < k_end) fill_x(k0 + SLAB);
        sg::cp_async_commit();
        const float *ws = ring + stage * Z::W_ELEMS + (lane & 3) * 2 * Z::W_PITCH + group * 32 + (lane >> 2) * 4;
        const bf16 *xa = xs + (lane & 15) * Z::X_PITCH + (lane >> 4) * 8;
#pragma unroll
        for (int kh = 0; kh < SLAB / PIECES; kh += 16) {
            const int kk = piece * (SLAB / PIECES) + kh;
            uint32_t fb[2][3][4];   // [k, k + 8][part][tile]
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                float x[4], y[4];
                load4(ws + (kk + 8 * d) * Z::W_PITCH, x);
                load4(ws + (kk + 8 * d + 1) * Z::W_PITCH, y);
                parts_of_pairs(x, y, fb[d]);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float d[4][4];
#pragma unroll
                for (int pa = 2; pa >= 0; --pa) {
                    uint32_t fa[4];
                    ldmatrix4<false>(fa, xa + pa * Z::X_PLANE + m * 16 * Z::X_PITCH + kk);
#pragma unroll
                    for (int pb = 2 - pa; pb >= 0; --pb)
#pragma unroll
                        for (int t = 0; t < 4; ++t)
                            if (pa == 2)
                                mma16816_first(d[t], fa, fb[0][pb][t], fb[1][pb][t]);
                            else
                                mma16816(d[t], fa, fb[0][pb][t], fb[1][pb][t]);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[m][t][e] += d[t][e];
            }
        }
        stage ^= 1;
    }
    // the pieces of the slabs' k in order, then out
    auto place = [&](int p, int m, int t, int e) {
        const int at = ((p - 1) * MT * 16 + (m * 4 + t) * 4 + e) * 128 + group * 32 + lane;
        return ring + (SG_IN_RANGE(at >= 0 && at < STAGES * Z::W_ELEMS) ? at : 0);
    };
    __syncthreads();
    if (piece > 0) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) *place(piece, m, t, e) = sum[m][t][e];
    }
    __syncthreads();
    if (piece > 0) return;
    float *out = partial + (long long)q * w.M * w.N;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = m * 16 + (lane >> 2) + (e / 2) * 8, j = n0 + group * 32 + 4 * ((lane & 3) * 2 + (e & 1));
            float v[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                v[t] = sum[m][t][e];
#pragma unroll
                for (int p = 1; p < PIECES; ++p) v[t] += *place(p, m, t, e);
            }
            if (i >= w.M) continue;
            if (w.N % 4 == 0 && j < w.N) {
                *reinterpret_cast<float4 *>(out + (long long)i * w.N + j) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (j + t < w.N) out[(long long)i * w.N + j + t] = v[t];
            }
        }
}

template <int MT>
__global__ void __launch_bounds__(RANK_THREADS, 2)
    few_rows_kernel(RowsWork w, Rows<float> X, const float *W, long long ldw, bool w_wide) {
    extern __shared__ __align__(16) unsigned char smem_rows[];
    sg::launch_dependents();
    few_rows<MT>(w, int(blockIdx.x), X, W, ldw, w_wide, w.partial, smem_rows);
}

// ------------------------------------------------------------------ the rest
// Y from the partial sums: a block to 256 columns of a row (8 to a lane), its 8 warps to
// the ranges and the rank, whose terms they share out; the warps' sums are added in
// order.  The first block of a row also writes H.  WIDE: rows of everything but the
// partial sums can be read eight elements at a time; `p_wide` the same of those.  EARLY, for
// grids of up to two blocks to an SM: the first terms of the rank are read before the sums
// are there (4 x 4096 x 4096 bfloat16 15.4 -> 14.4 us; 64 rows, of more blocks, 21.5 -> 23).
template <class T, bool WIDE, bool EARLY>
__global__ void __launch_bounds__(256)
    few_rows_finish_kernel(RowsWork w, Stack<const T> V, Adapters ad, const T *bias, bool p_wide, float *H, long long ldh,
                           T *Y, long long ldy) {
    __shared__ float S[128];
    __shared__ __align__(16) float sums[8][256];
    const int i = blockIdx.y, n0 = blockIdx.x * 256, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int j = n0 + lane * 8;
    if (!SG_IN_RANGE(i < w.M && n0 < w.N && (ad.L == 0 || ad.R <= 128))) return;
    const int a = ad.of_row(i), rank = a < 0 ? 0 : ad.rank(a);
    const float scale = a < 0 ? 0.0f : ad.scale(a);
    float x[8] = {}, v[8];
    auto read = [&](auto *p, bool eight, float (&v)[8]) {   // columns j .. j + 7
        if (eight && j + 8 <= w.N) {
            load8(p + j, v);
        } else {
#pragma unroll
            for (int d = 0; d < 8; ++d) v[d] = j + d < w.N ? to_f32(p[j + d]) : 0.0f;
        }
    };
    // the call's inputs, before the sums are there
    const T *m = rank > 0 ? V.matrix(a) : nullptr;
    float first[2][8];
#pragma unroll
    for (int u = 0; u < 2; ++u)
        if (EARLY && warp + 8 * u < rank) read(m + (warp + 8 * u) * V.ld, WIDE, first[u]);
    if (bias && warp == 7) read(bias, WIDE, x);
    sg::wait_prerequisites();
    if (int(threadIdx.x) < ad.R && ad.L > 0) {
        const int r = threadIdx.x;
        float sum = 0.0f;
        if (r < rank) {
            const float *p = w.rank_partial + (long long)i * ad.R + r;
#pragma unroll 8
            for (int q = 0; q < w.rank_ranges; ++q) sum += p[(long long)q * w.M * ad.R];
        }
        if (H && blockIdx.x == 0) H[i * ldh + r] = sum;
        S[r] = r < rank ? sum * scale : 0.0f;
    }
    const float *p = w.partial + (long long)i * w.N;
    const long long plane = (long long)w.M * w.N;
#pragma unroll 2
    for (int q = warp; q < w.ranges; q += 8) {
        read(p + q * plane, p_wide, v);
#pragma unroll
        for (int d = 0; d < 8; ++d) x[d] += v[d];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u)
        if (EARLY && warp + 8 * u < rank)
#pragma unroll
            for (int d = 0; d < 8; ++d) x[d] = fmaf(S[warp + 8 * u], first[u][d], x[d]);
#pragma unroll 4
    for (int r = warp + (EARLY ? 16 : 0); r < rank; r += 8) {
        read(m + r * V.ld, WIDE, v);
#pragma unroll
        for (int d = 0; d < 8; ++d) x[d] = fmaf(S[r], v[d], x[d]);
    }
    *reinterpret_cast<float4 *>(&sums[warp][lane * 8]) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(&sums[warp][lane * 8 + 4]) = make_float4(x[4], x[5], x[6], x[7]);
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += sums[k][threadIdx.x];
    if (n0 + int(threadIdx.x) < w.N) Y[(long long)i * ldy + n0 + threadIdx.x] = from_f32<T>(s);
}

}  // namespace sgl
