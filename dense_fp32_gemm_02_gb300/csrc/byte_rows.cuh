// byte_rows.cuh -- the product of int8 matrices for one to four rows: W streamed once through the integer
// units, and rows of the type brought to 8 bits on the way.
//
// Bound by reading W; at one row by the launch and the latencies around that too, so the call is this one
// kernel.  A block has 128 columns (or 64) and a range of the contraction; the ranges of a tile, up to 8, are a
// cluster.  A thread has 64 bytes of W on their way at a time, four k of 8 columns, twice (four rows: of 4
// columns, four times, as its registers hold 16 sums and those).  It turns each four words into four of
// four k (eight byte permutations) and adds products of four k in one instruction: 0.75 instructions to
// a byte of W for a row, 0.25 more for each other.  W's first step is on its way while the block finds the
// rows' largest magnitudes (each block of all of K: the rows are short and in L2) and lays its range of q
// in shared memory.  The sums are int32: a warp's by halving exchanges, the warps' and the ranges' in
// shared memory, each block finishing a share of the columns.
//
// us, q and its scale given, with the share of the copy's bandwidth: one row, 4096 x 4096 6.3 (40 %), 8192 x
// 8192 13.5 (74 %), 16384 x 8192 23.6 (85 %), 8191 x 8191 18.7, 1024 x 1024 2.9; rows of bfloat16 take
// 0.4 to 2 more.  Columns 16 to a thread took 7.5, 14.5, 24.2, 20.7 and 3.8; the loads behind a test
// each, in place of one for the four, 6.4, 15.5, 27.4, 41 and 3.2; the next step's loads ahead of this one's
// products 6.4, 15.0, 26.3.
#pragma once

#include "linear8.cuh"
#include "rows8.cuh"

namespace sgl {

constexpr int ROWS_THREADS = 512, ROWS_WARPS = ROWS_THREADS / 32;
constexpr int ROWS_RANGE = 8192;   // at most
__host__ __device__ constexpr int rows_step(int tile) { return ROWS_THREADS * 64 / tile; }   // k of a block's step, 64 bytes to a thread

template <class T>
struct ByteRows {
    int M, N, K, ranges, range;   // range: a multiple of the step
    const T *X;                   // or q and scale
    const signed char *q, *W;
    const float *scale, *wscale;
    const T *bias;
    T *Y;
    long long ldx, ldq, ldw, ldy;
};

template <int ROWS, int TILE>
constexpr size_t byte_rows_smem(int range) { return size_t(ROWS) * (ROWS_WARPS * TILE * 4 + range); }

// Four rows of 4 * WORDS bytes from p on, of a matrix from `begin` to `end`, `rows` of them and `cols` of a
// row being the block's: aligned as they are, or of two aligned loads shifted into place; where those would
// leave the matrix, and where there are fewer rows, byte by byte.
template <int WORDS, bool WIDE>
__device__ __forceinline__ void take_columns(const signed char *p, long long ld, const signed char *begin, const signed char *end,
                                             int rows, int cols, uint32_t (&w)[4][WORDS]) {
    using V = std::conditional_t<WORDS == 4, uint4, std::conditional_t<WORDS == 2, uint2, uint32_t>>;
    constexpr int BYTES = 4 * WORDS;
    if (rows >= 4 && p - (WIDE ? 0 : BYTES - 1) >= begin && p + 3 * ld + (WIDE ? BYTES : 2 * BYTES) <= end) {
        V v[4][WIDE ? 1 : 2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const signed char *at = p + i * ld;
            if constexpr (WIDE) {
                v[i][0] = __ldcs(reinterpret_cast<const V *>(at));
            } else {
                const V *down = reinterpret_cast<const V *>(reinterpret_cast<uintptr_t>(at) & ~uintptr_t(BYTES - 1));
                v[i][0] = down[0], v[i][1] = down[1];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (WIDE) {
                memcpy(w[i], v[i], BYTES);
            } else {
                uint32_t both[2 * WORDS];
                memcpy(both, v[i], 2 * BYTES);
                shift_bytes<1>(both, int(reinterpret_cast<uintptr_t>(p + i * ld) & (BYTES - 1)), w[i]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < WORDS; ++j) {
                w[i][j] = 0;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    if (i < rows && 4 * j + d < cols) w[i][j] |= uint32_t(static_cast<unsigned char>(p[i * ld + 4 * j + d])) << (8 * d);
            }
    }
}

template <class T, int ROWS, int TILE, bool WIDE>
__global__ void __launch_bounds__(ROWS_THREADS, 2) byte_rows_kernel(const ByteRows<T> a) {
    constexpr int WORDS = ROWS == 4 ? 1 : 2, COLS = 4 * WORDS, LANES = TILE / COLS, GROUP_K = ROWS_THREADS / LANES * 4;
    constexpr int STEP = rows_step(TILE), TIMES = STEP / GROUP_K, VALUES = ROWS * COLS, OUTPUTS = ROWS * TILE;
    extern __shared__ __align__(16) unsigned char byte_rows_shared[];
    int *parts = reinterpret_cast<int *>(byte_rows_shared);                      // of each warp: OUTPUTS
    uint32_t *rows = reinterpret_cast<uint32_t *>(parts + ROWS_WARPS * OUTPUTS);   // a range of q, row by row
    __shared__ int sums[OUTPUTS + 8];   // of the outputs that this block finishes: those of each range
    __shared__ uint32_t tops[ROWS_WARPS];
    __shared__ float scales[ROWS];
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    sg::wait_prerequisites();
    sg::launch_dependents();

    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int rank = int(blockIdx.x) % a.ranges, n0 = int(blockIdx.x) / a.ranges * TILE;
    const int k0 = rank * a.range, kn = min(a.range, a.K - k0), steps = (kn + STEP - 1) / STEP;
    const int col = n0 + (t % LANES) * COLS, group = t / LANES * 4;
    const bool sane = SG_IN_RANGE(kn > 0 && n0 < a.N && a.range <= ROWS_RANGE && a.M <= ROWS);
    const signed char *end = a.W + (a.K - 1) * a.ldw + a.N;
    auto load = [&](int step, uint32_t (&w)[TIMES][4][WORDS]) {
#pragma unroll
        for (int u = 0; u < TIMES; ++u) {
            const int k = step * STEP + u * GROUP_K + group;
            take_columns<WORDS, WIDE>(a.W + (k0 + k) * a.ldw + col, a.ldw, a.W, end, kn - k, a.N - col, w[u]);
        }
    };
    uint32_t w[TIMES][4][WORDS] = {};
    const bool busy = sane && col < a.N;
    if (busy) load(0, w);

    // ------------------------------------------------------------------ the rows' range of q
    constexpr int PER_ROW = ROWS_THREADS / ROWS, WARPS_PER_ROW = ROWS_WARPS / ROWS;   // threads to a row
    const int r = t / PER_ROW, first_k = t % PER_ROW * 4;
    const bool there = sane && r < a.M;
    const bool four = a.X ? (reinterpret_cast<uintptr_t>(a.X) & (4 * sizeof(T) - 1)) == 0 && a.ldx % 4 == 0
                          : (reinterpret_cast<uintptr_t>(a.q) & 3) == 0 && a.ldq % 4 == 0;
    const auto finite = [](float magnitude) { return magnitude < __uint_as_float(0x7f800000u); };
    auto values = [&](int k, float (&v)[4]) {
        const T *x = a.X + r * a.ldx + k;
        if (four && k + 4 <= a.K) {
            load4(x, v);
        } else {
#pragma unroll
            for (int d = 0; d < 4; ++d) v[d] = k + d < a.K ? to_f32(x[d]) : 0.0f;
        }
    };
    float largest = 0.0f, times = 0.0f;
    if (a.X) {
        uint32_t top = 0;
        if (there) {
#pragma unroll 4
            for (int k = first_k; k < a.K; k += PER_ROW * 4) {
                float v[4];
                values(k, v);
#pragma unroll
                for (int d = 0; d < 4; ++d) top = max(top, magnitude_bits(v[d]));
            }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) tops[warp] = top;
        __syncthreads();
        top = lane < WARPS_PER_ROW ? tops[warp / WARPS_PER_ROW * WARPS_PER_ROW + lane] : 0u;
        largest = __uint_as_float(__reduce_max_sync(0xffffffffu, top));
        if (largest >= LEAST_TOP && largest <= MOST_TOP) times = 127.0f / largest;
    }
    if (there && first_k == 0)
        scales[r] = !a.X                ? a.scale[r]
                    : times != 0.0f     ? largest / 127.0f
                    : finite(largest) ? float(double(largest) / 127.0) : __uint_as_float(0x7fc00000u);
    for (int k = first_k; k < steps * STEP; k += PER_ROW * 4) {
        uint32_t word = 0;
        if (!there || k >= kn) {
        } else if (!a.X) {
            const signed char *q = a.q + r * a.ldq + k0 + k;
            if (four && k + 4 <= kn) {
                word = *reinterpret_cast<const uint32_t *>(q);
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    if (k + d < kn) word |= uint32_t(static_cast<unsigned char>(q[d])) << (8 * d);
            }
        } else {
            float v[4];
            values(k0 + k, v);   // (what is behind the range, only at K's end, is 0)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                if (times != 0.0f) {
                    const float quotient = v[d] * times, q = whole(quotient);
                    v[d] = fabsf(quotient - q) > 0.5f - NEAR ? tie_exact(v[d], quotient, largest) : q;
                } else {   // zeros, an infinity or a NaN: no q; else in 64 bits
                    const bool keep = largest > 0.0f && finite(largest);
                    v[d] = keep ? float(__double2int_rn(127.0 * double(v[d]) / double(largest))) : 0.0f;
                }
            }
            word = pack_s8(v, 1.0f);
        }
        rows[(r * a.range + k) >> 2] = word;
    }
    __syncthreads();

    // ------------------------------------------------------------------ sums
    int sum[VALUES] = {};
    for (int step = 0; busy && step < steps; ++step) {
        if (step > 0) load(step, w);
#pragma unroll
        for (int u = 0; u < TIMES; ++u) {
            uint32_t x[ROWS];
#pragma unroll
            for (int i = 0; i < ROWS; ++i) x[i] = rows[(i * a.range + step * STEP + u * GROUP_K + group) >> 2];
#pragma unroll
            for (int j = 0; j < WORDS; ++j) {
                const uint32_t lo = __byte_perm(w[u][0][j], w[u][1][j], 0x5140), lo2 = __byte_perm(w[u][2][j], w[u][3][j], 0x5140);
                const uint32_t hi = __byte_perm(w[u][0][j], w[u][1][j], 0x7362), hi2 = __byte_perm(w[u][2][j], w[u][3][j], 0x7362);
                const uint32_t of[4] = {__byte_perm(lo, lo2, 0x5410), __byte_perm(lo, lo2, 0x7632),
                                        __byte_perm(hi, hi2, 0x5410), __byte_perm(hi, hi2, 0x7632)};
#pragma unroll
                for (int i = 0; i < ROWS; ++i)
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        sum[i * COLS + j * 4 + d] = __dp4a(int(of[d]), int(x[i]), sum[i * COLS + j * 4 + d]);
            }
        }
    }
    // the lanes of a column: each exchange leaves a lane half of its values, at the end LEFT from `first`
    constexpr int LEFT = OUTPUTS / 32, PAIR = LEFT < 4 ? 2 : 4;
    int first = 0;
#pragma unroll
    for (int o = 16, half = VALUES / 2; o >= LANES; o >>= 1, half /= 2) {
        const bool upper = (lane & o) != 0;
        first += upper ? half : 0;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const int mine = upper ? sum[i + half] : sum[i], other = upper ? sum[i] : sum[i + half];
            sum[i] = mine + __shfl_xor_sync(0xffffffffu, other, o);
        }
    }
#pragma unroll
    for (int i = 0; i < LEFT; i += PAIR) {
        const int f = first + i, at = f / COLS * TILE + (lane % LANES) * COLS + f % COLS;
        if constexpr (PAIR == 4)
            *reinterpret_cast<int4 *>(parts + warp * OUTPUTS + at) = make_int4(sum[i], sum[i + 1], sum[i + 2], sum[i + 3]);
        else
            *reinterpret_cast<int2 *>(parts + warp * OUTPUTS + at) = make_int2(sum[i], sum[i + 1]);
    }
    __syncthreads();
    // ------------------------------------------------------------------ outputs: `share` of them to a block
    const int share = (OUTPUTS + a.ranges - 1) / a.ranges;
    const int o = rank * share + t, m = o / TILE, n = n0 + o % TILE;
    const bool mine = sane && t < share && o < OUTPUTS && m < a.M && n < a.N;
    const float of = mine ? a.wscale[n] : 0.0f, add = mine && a.bias ? to_f32(a.bias[n]) : 0.0f;
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // all have begun
    if (t < OUTPUTS) {
        int s = 0;
#pragma unroll
        for (int i = 0; i < ROWS_WARPS; ++i) s += parts[i * OUTPUTS + t];
        const int owner = t / share;
        asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(
                         sg::dsmem_map(sg::smem_addr(&sums[rank * share + t - owner * share]), uint32_t(owner))), "r"(s) : "memory");
    }
    sg::cluster_barrier();
    if (!mine) return;
    int s = 0;
    for (int c = 0; c < a.ranges; ++c) s += sums[c * share + t];
    float y = float(s) * (scales[m] * of);
    y = a.bias ? y + add : y;   // (without a bias nothing is added: it would turn -0 into 0)
    a.Y[m * a.ldy + n] = from_f32<T>(y);
}

}  // namespace sgl
