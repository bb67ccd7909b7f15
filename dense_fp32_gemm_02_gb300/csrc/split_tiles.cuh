// split_tiles.cuh -- the gated block's two projections of float32 rows, 17 to 192 of them, W brought to three
// bfloat16 parts inside shared memory.
//
// Bound by reading W once: parts laid out first are written and read again, 2.5 times W's bytes more.  The
// rows are the MMA's narrow side: a tile is 128 columns of one of the two W (the MMA's M) by up to 64 rows of X (its
// N), whose parts are laid out before; a block has one tile and one range of the contraction, and writes its sums
// to partial[matrix][range][row][column] for pair_finish_kernel.  As in parts_gemm.cuh the six products go to two
// kinds of accumulators: the large ones to one that is taken to fp32 registers every 256 k while another fills, the
// small pairs to one of their own.
//
// 608 threads.  Warp 16 copies slabs of 64 k of W by TMA, two ahead (W whose rows are not 16-byte aligned: each
// team its own, four bytes at a time); warp 18 the same of X's parts, straight to where the MMA wants them.
// Warps 0 to 15 split W, in two teams, a slab and a stage to each, a thread eight columns at a time, and store them
// with the columns next to each other (128-byte swizzle).  Warp 17 issues the MMAs.  At the end warps 0 to 15 take
// the sums out, a lane to a column of W.
//
// us, whole call: 64 rows of 4096 x 4096 41.7 (3.2 TB/s; by warp-level MMAs that split what they read 95.9, by
// parts laid out first 114), 16 rows 40.7, 128 rows 70.7 (116); 64 rows of 4096 x 8192 72.6 (182), of
// 1024 x 1024 10.8 (17.8).  A slab takes an SM 1.0 us: splitting and storing 8192 elements, the 24 MMAs' reads of shared
// memory (0.6) and the stores beside them.  Four bytes at a time: 64 rows of 4096 x 4095 65.7 (one warp
// copying for both teams 118).
#pragma once

#include "gated.cuh"
#include "tiles.cuh"

namespace sgl {

constexpr int SPLIT_COLS = 128, SPLIT_ROWS = 64, SPLIT_STEP = 64, SPLIT_CHUNK = 4;   // (slabs to a chunk)
constexpr int SPLIT_CONVERTERS = 512, SPLIT_THREADS = SPLIT_CONVERTERS + 96;
constexpr int SPLIT_STAGES = 2, SPLIT_DEPTH = SPLIT_STAGES;   // of parts, of W's bytes: one of either to a team
constexpr uint32_t SPLIT_RAW = SPLIT_COLS * SPLIT_STEP * 4, SPLIT_W_PART = SPLIT_COLS * SPLIT_STEP * 2,
                   SPLIT_X_PART = SPLIT_ROWS * SPLIT_STEP * 2, SPLIT_STAGE = 3 * (SPLIT_W_PART + SPLIT_X_PART);
constexpr size_t SPLIT_SMEM = SPLIT_STAGES * SPLIT_STAGE + SPLIT_DEPTH * SPLIT_RAW + 1024 + 256;
static_assert(SPLIT_SMEM <= 232448, "shared memory of a block");

struct SplitWork {
    int M, N, K;
    int across, down, ranges, range;   // tiles of columns (of one matrix), of rows; range: a multiple of SPLIT_STEP
    int rows;                          // of a tile: a multiple of 16
    float *partial;
    unsigned long long timeout_ns;
};

// The W: maps of them, and for rows that the TMA does not read (WIDE false) the matrices.
struct SplitWeights {
    const float *p[2];
    long long ld[2];
};

template <bool WIDE>
__global__ void __launch_bounds__(SPLIT_THREADS, 1)
    split_tiles_kernel(const __grid_constant__ CUtensorMap mX, const __grid_constant__ CUtensorMap mG,
                       const __grid_constant__ CUtensorMap mU, const SplitWeights weights, const SplitWork w) {
    using namespace sg;
    using namespace sg::t3;
    constexpr int WARPS = SPLIT_CONVERTERS / 32, TEAM = SPLIT_CONVERTERS / SPLIT_STAGES;
    extern __shared__ unsigned char smem_split[];
    const uintptr_t base = (reinterpret_cast<uintptr_t>(smem_split) + 1023) & ~uintptr_t(1023);
    const uint32_t stages = smem_addr(reinterpret_cast<void *>(base)), raw = stages + SPLIT_STAGES * SPLIT_STAGE;
    uint64_t *full = reinterpret_cast<uint64_t *>(base + SPLIT_STAGES * SPLIT_STAGE + SPLIT_DEPTH * SPLIT_RAW);
    uint64_t *empty = full + SPLIT_STAGES;      // converters -> MMA, and back
    uint64_t *landed = empty + SPLIT_STAGES;    // W's copies -> converters
    uint64_t *taken = landed + SPLIT_DEPTH;     // and back
    uint64_t *acc_full = taken + SPLIT_DEPTH;   // MMA -> converters, [2]
    uint64_t *acc_empty = acc_full + 2;         // and back
    uint64_t *drain = acc_empty + 2;
    uint64_t *x_landed = drain + 1;             // X's copies -> MMA
    uint32_t *tmem_base = reinterpret_cast<uint32_t *>(x_landed + SPLIT_STAGES);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_base + 1);
    constexpr uint32_t SMALL = 2 * SPLIT_ROWS, TMEM = 256;   // columns: two large sums, the small pairs'

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < SPLIT_STAGES; ++s) {
            mbar_init(&full[s], WARPS / SPLIT_STAGES);
            mbar_init(&empty[s], 1);
            mbar_init(&x_landed[s], 1);
        }
        for (int d = 0; d < SPLIT_DEPTH; ++d) {
            mbar_init(&landed[d], WIDE ? 1 : TEAM);
            mbar_init(&taken[d], WARPS / SPLIT_STAGES);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], WARPS);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == WARPS + 1) tmem_alloc(tmem_base, TMEM);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    launch_dependents();   // (its call's second kernel; what it reads of the first one's it waits for below)
    const uint32_t taddr = *tmem_base;

    // a tile's rows are neighbours, whose W comes from L2, then the ranges, then the tiles of columns and the matrices
    const int d = int(blockIdx.x) % w.down, q = int(blockIdx.x) / w.down % w.ranges, n = int(blockIdx.x) / w.down / w.ranges;
    const bool second = n >= w.across;
    const int m0 = d * w.rows, n0 = (second ? n - w.across : n) * SPLIT_COLS;
    const int k0 = q * w.range, kn = min(w.range, w.K - k0);
    const bool sane = SG_IN_RANGE(n < 2 * w.across && kn > 0 && n0 < w.N && m0 < w.M && w.rows <= SPLIT_ROWS);
    const int slabs = sane ? (kn + SPLIT_STEP - 1) / SPLIT_STEP : 0, chunks = (slabs + SPLIT_CHUNK - 1) / SPLIT_CHUNK;
    auto give_up = [&](unsigned what) {
        atomicOr(&g_error_word, what);
        *abort_flag = 1;
    };
    float sum[16] = {};   // a lane's column, 16 rows of the tile to a group of four warps

    if (warp < WARPS) {
        // ================================================================ W to parts
        const int team = int(threadIdx.x) / TEAM, t = int(threadIdx.x) % TEAM;
        // eight columns of a k; units TEAM apart are 16 k on.  Lanes 4 to 7 of eight read the halves of their 32 bytes
        // in the other order, so that eight lanes meet all banks.
        const int chunk8 = t & 7, group = t >> 3 & 1, k = t >> 4, swap = t >> 2 & 1;
        const uint32_t from = raw + uint32_t(k * SPLIT_COLS * 4 + group * 256 + chunk8 * 32);
        const uint32_t to = stages + uint32_t(team) * SPLIT_STAGE + uint32_t(group) * uint32_t(sgp::GROUP_BYTES) + uint32_t(k * 128) +
                            uint32_t((chunk8 ^ (k & 7)) << 4);
        const int quarter = warp & 3, r0 = (warp >> 2) * 16;
        const uint32_t lanes = taddr + uint32_t(r0) + (uint32_t(quarter * 32) << 16);
        auto add = [&](uint32_t acc) {
            if (r0 >= w.rows) return;
            float v[16];
            tmem_add16(lanes + acc, v, false);
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[i] += v[i];
        };
        auto take_out = [&](int chunk) {
            bool ok = mbar_wait(&acc_full[chunk & 1], uint32_t(chunk >> 1) & 1u, w.timeout_ns);
            if (!ok && !*abort_flag) give_up(ERR_FULL_WAIT);
            if (!__all_sync(0xffffffffu, ok)) return false;
            tc_fence_after();
            add(uint32_t(chunk & 1) * SPLIT_ROWS);
            if (chunk == chunks - 1) add(SMALL);   // (complete with the last chunk)
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[chunk & 1]);
            return true;
        };
        // rows that the TMA does not read: a team copies its own next slab, a warp eight k, a lane every 32nd column, zeros
        // outside the matrix
        auto copy = [&](int s) {
            const int first = k0 + s * SPLIT_STEP + (t >> 5) * 8;
            const float *W = weights.p[second];
            const long long ld = weights.ld[second];
            const uint32_t at = raw + uint32_t(team) * SPLIT_RAW + uint32_t(((t >> 5) * 8 * SPLIT_COLS + lane) * 4);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < SPLIT_COLS; j += 32) {
                    const int c = n0 + j + lane;
                    const bool in = first + i < w.K && c < w.N;
                    cp_async4(at + uint32_t((i * SPLIT_COLS + j) * 4), in ? W + (first + i) * ld + c : W, in ? 4u : 0u);
                }
            cp_async_arrive(smem_addr(&landed[team]));
        };
        if (!WIDE && team < slabs) copy(team);
        int taken_out = 0;
        bool ok = true;
        for (int s = team, use = 0; s < slabs; s += SPLIT_STAGES, ++use) {
            const int depth = team;
            ok = mbar_wait(&empty[team], (uint32_t(use) & 1u) ^ 1u, w.timeout_ns) &&
                 mbar_wait(&landed[depth], uint32_t(s / SPLIT_DEPTH) & 1u, w.timeout_ns);
            if (!ok && !*abort_flag) give_up(ERR_FULL_WAIT);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            uint4 v[SPLIT_STEP / 16][2];
#pragma unroll
            for (int i = 0; i < SPLIT_STEP / 16; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    v[i][h] = lds_words(from + uint32_t(depth) * SPLIT_RAW + uint32_t(i * 16 * SPLIT_COLS * 4 + (h ^ swap) * 16));
            if (!WIDE && s + SPLIT_STAGES < slabs) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&taken[depth]);
                ok = mbar_wait(&taken[depth], uint32_t(use) & 1u, w.timeout_ns);
                if (!ok && !*abort_flag) give_up(ERR_EMPTY_WAIT);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                copy(s + SPLIT_STAGES);
            }
#pragma unroll
            for (int i = 0; i < SPLIT_STEP / 16; ++i) {
                const uint4 lo = swap ? v[i][1] : v[i][0], hi = swap ? v[i][0] : v[i][1];
                const uint32_t x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                float part[8][3];
#pragma unroll
                for (int e = 0; e < 8; ++e) split_parts(__uint_as_float(x[e]), part[e]);
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    sts_words(to + uint32_t(p) * SPLIT_W_PART + uint32_t(i * 16 * 128), pack_exact(part[0][p], part[1][p]),
                              pack_exact(part[2][p], part[3][p]), pack_exact(part[4][p], part[5][p]), pack_exact(part[6][p], part[7][p]));
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the MMA reads what was written
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&full[team]);
                if (WIDE) mbar_arrive(&taken[depth]);
            }
            // a chunk that is done, while the MMAs of this one go on
            if (taken_out < s / SPLIT_CHUNK && !(ok = take_out(taken_out++))) break;
        }
        while (ok && taken_out < chunks) ok = take_out(taken_out++);
        if (!WIDE) cp_async_wait_all();
    } else if (warp == WARPS) {
        // ================================================================ W's copies
        int depth = 0, issued = 0;
        uint32_t phase = 0;
        for (; WIDE && issued < slabs; ++issued) {
            if (!__all_sync(0xffffffffu, mbar_wait(&taken[depth], phase ^ 1u, w.timeout_ns))) {
                give_up(ERR_EMPTY_WAIT);
                break;
            }
            const uint32_t bar = smem_addr(&landed[depth]), to = raw + uint32_t(depth) * SPLIT_RAW;
            const int k = k0 + issued * SPLIT_STEP;
            if (elect_one()) {
                mbar_arrive_expect_tx_at(bar, SPLIT_RAW);
                tma_load_2d_at(to, second ? &mU : &mG, bar, n0, k);
            }
            __syncwarp();
            if (++depth == SPLIT_DEPTH) depth = 0, phase ^= 1u;
        }
        for (int i = max(0, issued - SPLIT_DEPTH); i < issued; ++i)   // what is in flight lands before the block ends
            if (!mbar_wait(&landed[i % SPLIT_DEPTH], uint32_t(i / SPLIT_DEPTH) & 1u, drain_limit_ns(w.timeout_ns))) {
                atomicOr(&g_error_word, ERR_DRAIN_WAIT);
                break;
            }
    } else if (warp == WARPS + 2) {
        // ================================================================ copies of X's parts
        wait_prerequisites();
        const uint32_t bytes = uint32_t(w.rows) * SPLIT_STEP * 2;
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        for (; issued < slabs; ++issued) {
            if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1u, w.timeout_ns))) {
                give_up(ERR_EMPTY_WAIT);
                break;
            }
            const uint32_t bar = smem_addr(&x_landed[stage]), at = stages + uint32_t(stage) * SPLIT_STAGE + 3 * SPLIT_W_PART;
            if (elect_one()) {
                mbar_arrive_expect_tx_at(bar, 3 * bytes);
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    tma_load_3d_at(at + uint32_t(p) * SPLIT_X_PART, &mX, bar, k0 + issued * SPLIT_STEP, m0, p);
            }
            __syncwarp();
            if (++stage == SPLIT_STAGES) stage = 0, phase ^= 1u;
        }
        for (int i = max(0, issued - SPLIT_STAGES); i < issued; ++i)
            if (!mbar_wait(&x_landed[i % SPLIT_STAGES], uint32_t(i / SPLIT_STAGES) & 1u, drain_limit_ns(w.timeout_ns))) {
                atomicOr(&g_error_word, ERR_DRAIN_WAIT);
                break;
            }
    } else {
        // ================================================================ MMA issuer
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (uint32_t(w.rows >> 3) << 17) | (uint32_t(SPLIT_COLS >> 4) << 24);
        int stage = 0, s = 0;
        uint32_t phase = 0;
        for (; s < slabs; ++s) {
            const int chunk = s / SPLIT_CHUNK;
            const bool first = s % SPLIT_CHUNK == 0;
            if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase, w.timeout_ns) && mbar_wait(&x_landed[stage], phase, w.timeout_ns) &&
                                             (!first || mbar_wait(&acc_empty[chunk & 1], (uint32_t(chunk >> 1) & 1u) ^ 1u, w.timeout_ns)))) {
                give_up(ERR_FULL_WAIT);
                break;
            }
            tc_fence_after();
            const uint32_t acc = taddr + uint32_t(chunk & 1) * SPLIT_ROWS;
            const uint32_t sw = stages + uint32_t(stage) * SPLIT_STAGE, sx = sw + 3 * SPLIT_W_PART;
            if (elect_one()) {
                auto mma = [&](uint32_t to, int qw, int qx, int kk, bool accumulate) {
                    mma_half(to, sgp::part_desc<true>(sw + uint32_t(qw) * SPLIT_W_PART, kk),
                             sgp::part_desc<false>(sx + uint32_t(qx) * SPLIT_X_PART, kk), idesc, accumulate);
                };
#pragma unroll
                for (int kk = 0; kk < SPLIT_STEP / 16; ++kk) {
                    bool fresh = s == 0 && kk == 0;
#pragma unroll
                    for (int qw = 2; qw >= 0; --qw)
#pragma unroll
                        for (int qx = 2; qx >= 0; --qx)
                            if (qw + qx > 0 && qw + qx <= 2) {
                                mma(taddr + SMALL, qw, qx, kk, !fresh);
                                fresh = false;
                            }
                    mma(acc, 0, 0, kk, !first || kk > 0);
                }
                mma_commit(&empty[stage]);
                if (s % SPLIT_CHUNK == SPLIT_CHUNK - 1 || s == slabs - 1) mma_commit(&acc_full[chunk & 1]);
            }
            if (++stage == SPLIT_STAGES) stage = 0, phase ^= 1u;
        }
        if (s < slabs) {   // given up: no MMA may still run when the block ends
            if (elect_one()) mma_commit(drain);
            if (!mbar_wait(drain, 0u, drain_limit_ns(w.timeout_ns))) atomicOr(&g_error_word, ERR_DRAIN_WAIT);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (sane && !*abort_flag && warp < WARPS) {
        const int r0 = (warp >> 2) * 16, column = n0 + (warp & 3) * 32 + lane;
        float *at = w.partial + ((second ? (long long)w.ranges : 0LL) + q) * w.M * w.N + (long long)(m0 + r0) * w.N + column;
        const int rows = min(w.rows, w.M - m0) - r0;
        if (column < w.N)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < rows) at[(long long)i * w.N] = sum[i];
    }
    if (warp == WARPS + 1) {
        __syncwarp();
        tmem_dealloc(taddr, TMEM);
    }
}

}  // namespace sgl
