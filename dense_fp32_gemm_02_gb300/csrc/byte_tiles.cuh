// byte_tiles.cuh -- the product of int8 matrices of up to 256 rows to a tile on the tensor cores, W brought
// to float16 inside shared memory.
//
// Bound by reading W once.  The rows are the MMA's narrow side: a tile is 128 columns of W (the MMA's M) by
// up to 256 rows of X (its N), and a block has one tile and one range of the contraction.  The ranges of a
// tile, up to 8, are a cluster, whose blocks add each other's sums as int32 and share the rows out.
// Every int8 is exactly a float16 and a sum of 1024 products of two is at most 2^24, so an fp32
// accumulator holds it exactly; every 1024 k it goes to int32 registers, while the next one fills.
//
// 576 threads.  Warp 16 copies slabs of 64 k of both matrices' bytes by TMA, several ahead.  Warps 0 to
// 15 turn them into float16 (a byte plus 128 under the exponent of 1024, less 1152: five instructions
// for four) and store them where the MMA wants them (128-byte swizzle: W with its columns, X with its k
// next to each other), a thread 16 bytes at a time, in teams, a slab and a stage to each.  Warp 17
// issues the MMAs.  At the end warps 0 to 15 take the accumulators out, a lane to a column of W.
//
// Measured with parts left out: at 64 x 8192 x 8192 (30 us) the converting warps' steps, mostly
// latency, set the pace (0.36 us a slab on an SM, of which loads, stores, conversion and MMAs each save under a
// tenth); small calls are 5 us of launch, hand-overs and the cluster's sums.  Reading the bytes straight
// into registers, with the freed memory for more stages, took 12.0 us for 11.9 at 64 x 4096 x 4096
// and 24.9 for 20.0 at 256 rows.
#pragma once

#include "linear8.cuh"
#include "tiles.cuh"

namespace sgl {

constexpr int TILE_COLS = 128, TILE_CHUNK = 1024, TILE_CONVERTERS = 512, TILE_THREADS = TILE_CONVERTERS + 64;
constexpr int MOST_CLUSTER = 8;

struct TileWork {
    int M, N, K;
    int across, down, ranges, range;   // tiles of columns, of rows; range: a multiple of 128
    int rows;                          // of a tile: a multiple of 16
    unsigned long long timeout_ns;
};

// ROWS: of a tile at most.
template <int ROWS>
struct ByteTile {
    static constexpr int STEP = 64;                                       // k of a slab
    static constexpr int W_RAW = TILE_COLS * STEP, X_RAW = ROWS * STEP, RAW = W_RAW + X_RAW;
    static constexpr int TEAMS = ROWS <= 128 ? 4 : 2, TEAM = TILE_CONVERTERS / TEAMS;
    static constexpr int W_EACH = W_RAW / 16 / TEAM, X_EACH = X_RAW / 16 / TEAM;   // units of 16 bytes, to a thread
    static constexpr int STAGES = TEAMS, STAGE = 2 * RAW;
    static constexpr int DEPTH = ROWS == 32 ? 12 : ROWS == 64 ? 8 : ROWS == 128 ? 5 : 4;
    static constexpr size_t SMEM = size_t(STAGES) * STAGE + size_t(DEPTH) * RAW + 1024 + 512;
    static constexpr uint32_t TMEM = 2 * ROWS;                            // two accumulators
    static constexpr int PER_CHUNK = TILE_CHUNK / STEP, GROUPS = ROWS > 64 ? ROWS / 64 : 1;
    static_assert(SMEM <= 232448, "shared memory of a block");
    static_assert(ROWS * TILE_COLS * 4 <= STAGES * STAGE + DEPTH * RAW, "the sums take their place");
};

// Four int8 as two words of float16.
__device__ __forceinline__ uint2 halves_of(uint32_t w) {
    w ^= 0x80808080u;
    const uint32_t lo = __byte_perm(w, 0x64646464u, 0x4140), hi = __byte_perm(w, 0x64646464u, 0x4342);
    uint2 out;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(out.x) : "r"(lo), "r"(0x64806480u));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(out.y) : "r"(hi), "r"(0x64806480u));
    return out;
}
template <class T, int ROWS>
__global__ void __launch_bounds__(TILE_THREADS, 1)
    byte_tiles_kernel(const __grid_constant__ CUtensorMap mX, const __grid_constant__ CUtensorMap mW, const TileWork w,
                      const float *scale, const float *wscale, const T *bias, T *Y, long long ldy) {
    using Z = ByteTile<ROWS>;
    using namespace sg;
    using namespace sg::t3;
    constexpr int WARPS = TILE_CONVERTERS / 32;
    extern __shared__ unsigned char smem_tiles[];
    const uintptr_t base = (reinterpret_cast<uintptr_t>(smem_tiles) + 1023) & ~uintptr_t(1023);
    const uint32_t stages = smem_addr(reinterpret_cast<void *>(base)), raw = stages + Z::STAGES * Z::STAGE;
    uint64_t *full = reinterpret_cast<uint64_t *>(base + Z::STAGES * Z::STAGE + Z::DEPTH * Z::RAW);
    uint64_t *empty = full + Z::STAGES;       // converters -> MMA and back
    uint64_t *landed = empty + Z::STAGES;     // copies -> converters
    uint64_t *taken = landed + Z::DEPTH;      // and back
    uint64_t *acc_full = taken + Z::DEPTH;    // MMA -> converters, [2]
    uint64_t *acc_empty = acc_full + 2;       // and back
    uint64_t *drain = acc_empty + 2;
    uint32_t *tmem_base = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_base + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < Z::STAGES; ++s) {
            mbar_init(&full[s], WARPS / Z::TEAMS);
            mbar_init(&empty[s], 1);
        }
        for (int d = 0; d < Z::DEPTH; ++d) {
            mbar_init(&landed[d], 1);
            mbar_init(&taken[d], WARPS / Z::TEAMS);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], WARPS);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == WARPS + 1) {
        tmem_alloc(tmem_base, Z::TMEM);
    } else if (warp == WARPS && lane == 0) {
        tma_prefetch_desc(&mX);
        tma_prefetch_desc(&mW);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wait_prerequisites();
    launch_dependents();
    const uint32_t taddr = *tmem_base;

    // a tile's ranges are neighbours (a cluster), then the tiles of the same columns, whose W comes from L2
    const int q = int(blockIdx.x) % w.ranges, tile = int(blockIdx.x) / w.ranges;
    const int m0 = (tile % w.down) * w.rows, n0 = (tile / w.down) * TILE_COLS;
    const int rows = min(w.rows, (w.M - m0 + 15) & ~15);   // of the MMA
    const int k0 = q * w.range, kn = min(w.range, w.K - k0);
    const bool sane = SG_IN_RANGE(kn > 0 && n0 < w.N && m0 < w.M && rows <= ROWS && w.rows <= ROWS);
    const int slabs = sane ? (kn + Z::STEP - 1) / Z::STEP : 0;
    auto give_up = [&](unsigned what) {
        atomicOr(&g_error_word, what);
        *abort_flag = 1;
    };
    const int col = n0 + lane * 4;   // of the output, a warp to a row
    float of[4] = {}, add[4] = {}, row_scale = 0.0f;   // (lane i: of the warp's i-th row)
    int sum[Z::GROUPS][16];          // the tile's: a lane's column, 16 rows of each 64

    if (warp < WARPS) {
        // ================================================================ bytes to float16
#pragma unroll
        for (int d = 0; d < 4; ++d) {   // (early: they are needed at the end)
            if (col + d < w.N) of[d] = wscale[col + d];
            if (bias && col + d < w.N) add[d] = to_f32(bias[col + d]);
        }
        const long long own = m0 + q + (warp + lane * WARPS) * (long long)w.ranges;
        if (own < w.M) row_scale = scale[own];
        // where a unit's 16 values go in the team's stage: two 16-byte chunks of a 128-byte line, swizzled
        constexpr int TEAM = Z::TEAM;
        const int team = int(threadIdx.x) / TEAM, t = int(threadIdx.x) % TEAM;
        // W: 16 columns of a k, of two groups of 64 columns; X: 16 k of a row; units TEAM apart lie in the same place of
        // other lines.  (Four threads to a line's bytes and the next four to the next line's: their chunks, all
        // even ones, are swizzled to even and to odd places.)
        const int wk = ((t >> 2) & 7) | (t >> 6) << 3, wg = (t >> 5) & 1, xm = t >> 2, c = t & 3;
        const uint32_t stage = stages + uint32_t(team * Z::STAGE);
        const uint32_t w_line = stage + uint32_t(wg * int(sgp::GROUP_BYTES) + wk * 128), x_line = stage + uint32_t(2 * Z::W_RAW + xm * 128);
        const uint32_t w_to = w_line + uint32_t((2 * c ^ (wk & 7)) << 4), w_to1 = w_line + uint32_t(((2 * c + 1) ^ (wk & 7)) << 4);
        const uint32_t x_to = x_line + uint32_t((2 * c ^ (xm & 7)) << 4), x_to1 = x_line + uint32_t(((2 * c + 1) ^ (xm & 7)) << 4);
        const uint32_t w_from = uint32_t(wk * TILE_COLS + wg * 64 + c * 16), x_from = uint32_t(Z::W_RAW + xm * Z::STEP + c * 16);
        const int x_rows = rows - xm;   // from here on
        auto put = [&](uint32_t at, uint32_t at1, uint4 v) {
            const uint2 a = halves_of(v.x), b = halves_of(v.y), d = halves_of(v.z), e = halves_of(v.w);
            sts_words(at, a.x, a.y, b.x, b.y);
            sts_words(at1, d.x, d.y, e.x, e.y);
        };
        const int quarter = warp & 3, group = warp >> 2;
        auto take_out = [&](int chunk) {
            bool ok = mbar_wait(&acc_full[chunk & 1], uint32_t(chunk >> 1) & 1u, w.timeout_ns);
            if (!ok && !*abort_flag) give_up(ERR_FULL_WAIT);
            if (!__all_sync(0xffffffffu, ok)) return false;
            tc_fence_after();
#pragma unroll
            for (int g = 0; g < Z::GROUPS; ++g) {
                const int c = group * 16 + g * 64;
                if (c >= rows) break;
                float v[16];
                tmem_add16(taddr + uint32_t((chunk & 1) * ROWS + c) + (uint32_t(quarter * 32) << 16), v, false);
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[g][i] = __float2int_rn(v[i]) + (chunk > 0 ? sum[g][i] : 0);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[chunk & 1]);
            return true;
        };
        int taken_out = 0;
        bool ok = true;
        for (int s = team, use = 0; s < slabs; s += Z::TEAMS, ++use) {
            // (first use of a stage: parity 1 counts as complete)
            const int depth = s % Z::DEPTH;
            ok = mbar_wait(&empty[team], (uint32_t(use) & 1u) ^ 1u, w.timeout_ns) &&
                 mbar_wait(&landed[depth], uint32_t(s / Z::DEPTH) & 1u, w.timeout_ns);
            if (!ok && !*abort_flag) give_up(ERR_FULL_WAIT);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            const uint32_t from = raw + uint32_t(depth * Z::RAW);
            uint4 v[Z::W_EACH > Z::X_EACH ? Z::W_EACH : Z::X_EACH];
#pragma unroll
            for (int i = 0; i < Z::W_EACH; ++i) v[i] = lds_words(from + w_from + uint32_t(i * (TEAM / 8) * TILE_COLS));
#pragma unroll
            for (int i = 0; i < Z::W_EACH; ++i) put(w_to + uint32_t(i * (TEAM / 8) * 128), w_to1 + uint32_t(i * (TEAM / 8) * 128), v[i]);
#pragma unroll
            for (int i = 0; i < Z::X_EACH; ++i)
                if (i * (TEAM / 4) < x_rows) v[i] = lds_words(from + x_from + uint32_t(i * (TEAM / 4) * Z::STEP));
#pragma unroll
            for (int i = 0; i < Z::X_EACH; ++i)
                if (i * (TEAM / 4) < x_rows)
                    put(x_to + uint32_t(i * (TEAM / 4) * 128), x_to1 + uint32_t(i * (TEAM / 4) * 128), v[i]);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the MMA reads what was written
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&full[team]);
                mbar_arrive(&taken[depth]);
            }
            // a chunk that is done, while the MMAs of this one go on
            if (taken_out < s / Z::PER_CHUNK && !(ok = take_out(taken_out++))) break;
        }
        while (ok && taken_out * Z::PER_CHUNK < slabs) ok = take_out(taken_out++);
    } else if (warp == WARPS) {
        // ================================================================ copies
        int depth = 0, issued = 0;
        uint32_t phase = 0;
        for (; issued < slabs; ++issued) {
            if (!__all_sync(0xffffffffu, mbar_wait(&taken[depth], phase ^ 1u, w.timeout_ns))) {
                give_up(ERR_EMPTY_WAIT);
                break;
            }
            const uint32_t to = raw + uint32_t(depth * Z::RAW), bar = smem_addr(&landed[depth]);
            const int k = k0 + issued * Z::STEP;
            if (elect_one()) {
                mbar_arrive_expect_tx_at(bar, Z::RAW);
                tma_load_2d_at(to, &mW, bar, n0, k);
                tma_load_2d_at(to + Z::W_RAW, &mX, bar, k, m0);
            }
            __syncwarp();
            if (++depth == Z::DEPTH) depth = 0, phase ^= 1u;
        }
        for (int i = max(0, issued - Z::DEPTH); i < issued; ++i)   // what is in flight lands before the block ends
            if (!mbar_wait(&landed[i % Z::DEPTH], uint32_t(i / Z::DEPTH) & 1u, drain_limit_ns(w.timeout_ns))) {
                atomicOr(&g_error_word, ERR_DRAIN_WAIT);
                break;
            }
    } else {
        // ================================================================ MMA issuer
        const uint32_t idesc = (1u << 4) | (1u << 15) | (uint32_t(rows >> 3) << 17) | (uint32_t(TILE_COLS >> 4) << 24);
        const uint64_t desc_w = sgp::part_desc<true>(stages, 0), desc_x = sgp::part_desc<false>(stages + 2 * Z::W_RAW, 0);
        int stage = 0, s = 0;
        uint32_t phase = 0;
        for (; s < slabs; ++s) {
            const int chunk = s / Z::PER_CHUNK;
            const bool first = s % Z::PER_CHUNK == 0;
            if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase, w.timeout_ns) &&
                                             (!first || mbar_wait(&acc_empty[chunk & 1], (uint32_t(chunk >> 1) & 1u) ^ 1u, w.timeout_ns)))) {
                give_up(ERR_FULL_WAIT);
                break;
            }
            tc_fence_after();
            const uint32_t acc = taddr + uint32_t((chunk & 1) * ROWS);
            const uint64_t da = desc_w + uint64_t(stage * (Z::STAGE >> 4)), db = desc_x + uint64_t(stage * (Z::STAGE >> 4));
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < Z::STEP / 16; ++kk) mma_half(acc, da + kk * (2048 >> 4), db + kk * (32 >> 4), idesc, !first || kk > 0);
                mma_commit(&empty[stage]);
                if (s % Z::PER_CHUNK == Z::PER_CHUNK - 1 || s == slabs - 1) mma_commit(&acc_full[chunk & 1]);
            }
            if (++stage == Z::STAGES) stage = 0, phase ^= 1u;
        }
        if (s < slabs) {   // given up: no MMA may still run when the block ends
            if (elect_one()) mma_commit(drain);
            if (!mbar_wait(drain, 0u, drain_limit_ns(w.timeout_ns))) atomicOr(&g_error_word, ERR_DRAIN_WAIT);
        }
    }
    __syncthreads();
    const bool good = sane && !*abort_flag;
    const uint32_t sums = stages;   // rows x 128 int32 in the place of all that, which nothing reads any more
    if (good && warp < WARPS) {
#pragma unroll
        for (int g = 0; g < Z::GROUPS; ++g) {
            const int c = (warp >> 2) * 16 + g * 64;
            if (c >= rows) break;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(sums + uint32_t((c + i) * TILE_COLS + (warp & 3) * 32 + lane) * 4),
                             "r"(sum[g][i]) : "memory");
        }
    }
    // ================================================================ the cluster's sums, a warp to a row
    cluster_barrier();
    if (good && warp < WARPS) {
        const bool wide = (reinterpret_cast<uintptr_t>(Y) & (4 * sizeof(T) - 1)) == 0 && ldy % 4 == 0 && col + 4 <= w.N;
        for (int r = q + warp * w.ranges, i = 0; r < rows; r += WARPS * w.ranges, ++i) {   // (i < 16)
            const long long m = m0 + r;
            if (m >= w.M) break;
            const float of_row = __shfl_sync(0xffffffffu, row_scale, i);
            int s[4] = {};
#pragma unroll 4
            for (int c = 0; c < w.ranges; ++c) {
                uint32_t x[4];
                asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                             : "r"(dsmem_map(sums + uint32_t(r * TILE_COLS + lane * 4) * 4, uint32_t(c))) : "memory");
#pragma unroll
                for (int d = 0; d < 4; ++d) s[d] += int(x[d]);
            }
            float y[4];
#pragma unroll
            for (int d = 0; d < 4; ++d) {   // (without a bias nothing is added: it would turn -0 into 0)
                y[d] = float(s[d]) * (of_row * of[d]);
                y[d] = bias ? y[d] + add[d] : y[d];
            }
            T *out = Y + m * ldy + col;
            if (wide) {
                store4(out, y);
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    if (col + d < w.N) out[d] = from_f32<T>(y[d]);
            }
        }
    }
    cluster_barrier();   // this block's sums have been read
    tc_fence_after();
    if (warp == WARPS + 1) {
        __syncwarp();
        tmem_dealloc(taddr, Z::TMEM);
    }
}

// Rows of bytes at any pitch as rows that are 16-byte aligned (what lies behind a row in its last 16
// is never read as the matrix's): a thread to 16 bytes, two aligned loads shifted into place, or, where those
// would leave the matrix, byte by byte.
static __global__ void __launch_bounds__(256)
    byte_pitch_kernel(const signed char *p, long long ld, int rows, int cols, Divisor per_row, signed char *out, long long pitch) {
    sg::wait_prerequisites();
    sg::launch_dependents();
    const long long total = (long long)rows * per_row.d, step = (long long)gridDim.x * 256;
    const bool small = total <= 0x7fffffffll;
    const signed char *end = p + (rows - 1) * ld + cols;
    for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < total; t += step) {
        const long long i = small ? (long long)per_row.quotient(unsigned(t)) : t / per_row.d;
        const int c = int(t - i * per_row.d) * 16;
        if (!SG_IN_RANGE(i < rows && c < cols && c + 16 <= pitch)) continue;
        const signed char *from = p + i * ld + c;
        const int shift = int(reinterpret_cast<uintptr_t>(from) & 15);
        uint32_t v[4];
        if (from - shift >= p && from - shift + 32 <= end) {
            const uint4 at[2] = {reinterpret_cast<const uint4 *>(from - shift)[0], reinterpret_cast<const uint4 *>(from - shift)[1]};
            uint32_t both[8];
            memcpy(both, at, 32);
            shift_bytes<1>(both, shift, v);
        } else {
            alignas(16) signed char x[16];
#pragma unroll
            for (int d = 0; d < 16; ++d) x[d] = c + d < cols ? from[d] : static_cast<signed char>(0);
            memcpy(v, x, 16);
        }
        *reinterpret_cast<uint4 *>(out + i * pitch + c) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

}  // namespace sgl
