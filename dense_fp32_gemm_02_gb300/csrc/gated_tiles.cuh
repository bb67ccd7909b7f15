// gated_tiles.cuh -- the gated block of up to 64 bfloat16 rows in one launch.
//
// Bound by reading both W once; at small sizes by launches and hand-overs, so the ranges of the contraction meet in
// a cluster instead of in memory.  The rows are the MMAs' narrow side: a tile is the same 128 columns of both W (the
// MMAs' M) by all rows (their N), G's and U's sums beside one another; the ranges of a tile, up to 8, are a
// cluster, whose blocks add each other's sums in order and share the rows out.
//
// 320 threads, two blocks to an SM: warp 8 copies slabs of 64 k by TMA, two or three ahead (32 KB of W each), warp 9
// issues the MMAs, warps 0 to 7 take the sums out, four of them G's and four U's, a lane to a column.  A sum
// stays in its accumulator for up to 8192 k, as in pair_gemm.cuh.
//
// us, bfloat16, SILU: 8 rows of 4096 x 8192 22.7 (5.9 TB/s), of 4096 x 4096 13.6, of 1024 x 1024 4.3; 64 rows 26.3,
// 19.4 and 6.1.  One row takes 0.1 to 0.5 less than 8.
#pragma once

#include "gated.cuh"
#include "tiles.cuh"

namespace sgl {

constexpr int GATED_COLS = 128, GATED_STEP = 64, GATED_WARPS = 8, GATED_THREADS = (GATED_WARPS + 2) * 32;
constexpr int GATED_CLUSTER = 8, GATED_RANGE = 8192;   // at most

struct GatedTileWork {
    int M, N, K;
    int across, ranges, range;   // range: a multiple of GATED_STEP
    int rows;                    // of the MMA: a multiple of 16
    unsigned long long timeout_ns;
};

// ROWS: at most.
template <int ROWS>
struct GatedTile {
    static constexpr uint32_t W_SLAB = 2 * sgp::GROUP_BYTES, STAGE = 2 * W_SLAB + ROWS * GATED_STEP * 2;
    static constexpr int STAGES = ROWS <= 32 ? 3 : 2;
    static constexpr size_t SMEM = size_t(STAGES) * STAGE + 1024 + 128;
    static constexpr uint32_t TMEM = 2 * ROWS;
    static_assert(2 * SMEM + 2048 <= 233472, "two blocks to an SM");
    static_assert(2 * ROWS * GATED_COLS * 4 <= STAGES * STAGE, "the sums take the slabs' place");
};

template <int ROWS>
__global__ void __launch_bounds__(GATED_THREADS, 2)
    gated_tiles_kernel(const __grid_constant__ CUtensorMap mX, const __grid_constant__ CUtensorMap mG,
                       const __grid_constant__ CUtensorMap mU, const GatedTileWork w, const PairOut<bf16> to) {
    using Z = GatedTile<ROWS>;
    using namespace sg;
    using namespace sg::t3;
    extern __shared__ unsigned char smem_gated[];
    const uintptr_t base = (reinterpret_cast<uintptr_t>(smem_gated) + 1023) & ~uintptr_t(1023);
    const uint32_t stages = smem_addr(reinterpret_cast<void *>(base));
    uint64_t *full = reinterpret_cast<uint64_t *>(base + Z::STAGES * Z::STAGE);
    uint64_t *empty = full + Z::STAGES;
    uint64_t *done = empty + Z::STAGES;
    uint64_t *drain = done + 1;
    uint32_t *tmem_base = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_base + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < Z::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == GATED_WARPS + 1) tmem_alloc(tmem_base, Z::TMEM);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wait_prerequisites();
    launch_dependents();
    const uint32_t taddr = *tmem_base;

    const int q = int(blockIdx.x) % w.ranges, n0 = int(blockIdx.x) / w.ranges * GATED_COLS;
    const int k0 = q * w.range, kn = min(w.range, w.K - k0);
    const bool sane = SG_IN_RANGE(kn > 0 && kn <= GATED_RANGE && n0 < w.N && w.M <= w.rows && w.rows <= ROWS);
    const int slabs = sane ? (kn + GATED_STEP - 1) / GATED_STEP : 0;
    auto give_up = [&](unsigned what) {
        atomicOr(&g_error_word, what);
        *abort_flag = 1;
    };

    if (warp == GATED_WARPS) {
        // ================================================================ copies
        const uint32_t bytes = 2 * Z::W_SLAB + uint32_t(w.rows) * GATED_STEP * 2;
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        for (; issued < slabs; ++issued) {
            if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1u, w.timeout_ns))) {
                give_up(ERR_EMPTY_WAIT);
                break;
            }
            const uint32_t at = stages + uint32_t(stage) * Z::STAGE, bar = smem_addr(&full[stage]);
            const int k = k0 + issued * GATED_STEP;
            if (elect_one()) {
                mbar_arrive_expect_tx_at(bar, bytes);
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    tma_load_3d_at(at + uint32_t(g) * sgp::GROUP_BYTES, &mG, bar, n0 + g * 64, k, 0);
                    tma_load_3d_at(at + Z::W_SLAB + uint32_t(g) * sgp::GROUP_BYTES, &mU, bar, n0 + g * 64, k, 0);
                }
                tma_load_3d_at(at + 2 * Z::W_SLAB, &mX, bar, k, 0, 0);
            }
            __syncwarp();
            if (++stage == Z::STAGES) stage = 0, phase ^= 1u;
        }
        for (int i = max(0, issued - Z::STAGES); i < issued; ++i)   // what is in flight lands before the block ends
            if (!mbar_wait(&full[i % Z::STAGES], uint32_t(i / Z::STAGES) & 1u, drain_limit_ns(w.timeout_ns))) {
                atomicOr(&g_error_word, ERR_DRAIN_WAIT);
                break;
            }
    } else if (warp == GATED_WARPS + 1) {
        // ================================================================ MMA issuer
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (uint32_t(w.rows >> 3) << 17) | (uint32_t(GATED_COLS >> 4) << 24);
        int stage = 0, s = 0;
        uint32_t phase = 0;
        for (; s < slabs; ++s) {
            if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase, w.timeout_ns))) {
                give_up(ERR_FULL_WAIT);
                break;
            }
            tc_fence_after();
            const uint32_t at = stages + uint32_t(stage) * Z::STAGE;
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < GATED_STEP / 16; ++kk)
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                        mma_half(taddr + uint32_t(m * ROWS), sgp::part_desc<true>(at + uint32_t(m) * Z::W_SLAB, kk),
                                 sgp::part_desc<false>(at + 2 * Z::W_SLAB, kk), idesc, s > 0 || kk > 0);
                mma_commit(&empty[stage]);
                if (s == slabs - 1) mma_commit(done);
            }
            if (++stage == Z::STAGES) stage = 0, phase ^= 1u;
        }
        if (s < slabs) {   // given up: no MMA may still run when the block ends
            if (elect_one()) mma_commit(drain);
            if (!mbar_wait(drain, 0u, drain_limit_ns(w.timeout_ns))) atomicOr(&g_error_word, ERR_DRAIN_WAIT);
        }
    } else if (sane) {
        // ================================================================ sums to shared memory: [matrix][row][column]
        const bool ok = mbar_wait(done, 0u, w.timeout_ns);
        if (!ok && !*abort_flag) give_up(ERR_FULL_WAIT);
        if (__all_sync(0xffffffffu, ok)) {
            tc_fence_after();
            const int quarter = warp & 3, m = warp >> 2;
            for (int r0 = 0; r0 < w.rows; r0 += 16) {
                float v[16];
                tmem_add16(taddr + uint32_t(m * ROWS + r0) + (uint32_t(quarter * 32) << 16), v, false);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(
                                     stages + uint32_t(((m * ROWS + r0 + i) * GATED_COLS + quarter * 32 + lane) * 4)), "f"(v[i]) : "memory");
            }
            tc_fence_before();
        }
    }
    // ================================================================ the cluster's sums, a warp to a row
    cluster_barrier();
    if (sane && !*abort_flag && warp < GATED_WARPS) {
        const int col = n0 + lane * 4, in = min(4, w.N - col);
        auto write = [&](bf16 *row, const float (&v)[4]) {
            if (in == 4 && (reinterpret_cast<uintptr_t>(row + col) & 7) == 0) {
                store4(row + col, v);
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    if (d < in) row[col + d] = from_f32<bf16>(v[d]);
            }
        };
        for (int r = q + warp * w.ranges; r < w.M; r += GATED_WARPS * w.ranges) {
            float s[2][4] = {};
#pragma unroll 4
            for (int c = 0; c < w.ranges; ++c)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float x[4];
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
                                 : "r"(dsmem_map(stages + uint32_t(((m * ROWS + r) * GATED_COLS + lane * 4) * 4), uint32_t(c))) : "memory");
#pragma unroll
                    for (int d = 0; d < 4; ++d) s[m][d] += x[d];
                }
            if (to.out) {
                write(to.out + r * to.ldo, s[0]);
                write(to.out1 + r * to.ldo1, s[1]);
            }
            with_act(to.act, [&](auto act) {
                float h[4];
#pragma unroll
                for (int d = 0; d < 4; d += 2) {
                    const float2 v = gate_value<bf16, decltype(act)::value>(make_float2(s[0][d], s[0][d + 1]));
                    h[d] = v.x * s[1][d], h[d + 1] = v.y * s[1][d + 1];
                }
                write(to.H + r * to.ldh, h);
            });
        }
    }
    cluster_barrier();   // this block's sums have been read
    tc_fence_after();
    if (warp == GATED_WARPS + 1) {
        __syncwarp();
        tmem_dealloc(taddr, Z::TMEM);
    }
}

}  // namespace sgl
