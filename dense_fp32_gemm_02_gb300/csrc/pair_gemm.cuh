// pair_gemm.cuh -- products of two matrices at once on pairs of SMs (tcgen05 `cta_group::2`): the
// gated block's two projections with their activation and product, its gradients, and the
// product of int8 matrices.
//
// What parts_gemm.cuh says of parts, of the accumulators' truncation and of the pipeline holds
// here too (copies, one issuing thread, eight epilogue warps; a 256 x 256 tile to a pair, 64 k to a
// slab, persistent; the abort protocol); this kernel has no rank side.  What differs:
//   GATE   each CTA of a pair loads one of the two matrices: a tile's accumulator has 128 columns of
//          G beside the same 128 of U, so that act(G) * U is made where both are, in registers.
//   SUM    the contraction runs over both pairs of operands, one after the other.
//   TWO    the tiles of both outputs are one list.
//   BYTES  an int8 is exactly a bfloat16, and sums of 1024 products of two are at most 2^24: exact
//          in the fp32 accumulator.  Every 1024 k it is taken to int32 registers, or every 2048 where
//          the rows' magnitudes keep such sums within 2^24 too (8192 x 4096 x 4096 over and over: 159 us for 182).
//          (The integer MMA of this GPU runs at a tenth of the bfloat16 one's rate.)
#pragma once

#include "gate.cuh"
#include "pair_gemm.h"
#include "parts_gemm.cuh"

namespace sgq {

using namespace sg;
using namespace sg::t3;
using sgp::BK;
using sgp::EPI_FLOATS;
using sgp::EPI_WARPS;
using sgp::GROUP_BYTES;
using sgp::PART_BYTES;
using sgp::part_desc;
using sgp::ROWS;
using sgp::SMEM_BYTES;
using sgp::SMEM_RING;
using sgp::THREADS;
using sgp::TILE;
using sgp::TMEM_COLUMNS;
using sgp::ACC_COLUMNS;

struct Params {
    int M, N;
    int tiles_m, tiles_n, group_m;   // tiles_n: of all outputs
    int tile_n;             // accumulator columns of a tile: 128 to 256
    int out_tiles;          // TWO: tiles_n of the first output
    int slabs, first_slabs; // of 64 k; SUM: of the first pair
    int splits, per_split;
    uint32_t slab_bytes;    // that a CTA loads of a slab
    float *partial;
    unsigned long long timeout_ns;
};

// Slabs of a chunk of the accumulation: see parts_gemm.cuh; BYTES 1024 k.
__host__ __device__ constexpr int chunk_slabs(bool several, bool bytes) { return bytes ? 16 : several ? 4 : sgp::LONG_CHUNK; }

__device__ __forceinline__ void sts_float(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// The work of a pair of CTAs, as sgp::Items; columns of an output are `cols` from col0, of which
// this CTA loads `load` from load0 of matrix `which`.
template <Mode MODE>
struct Work {
    int full, mine_full, mine;

    __device__ void init(const Params &p) {
        const int Q = gridDim.x / 2, q = blockIdx.x / 2;
        const int items = p.tiles_m * p.tiles_n * p.splits, tail = items % Q;
        full = (p.tile_n == TILE && p.splits == 1 && tail != 0 && 2 * tail <= Q) ? items - tail : items;
        const int halves = 2 * (items - full);
        mine_full = q < full ? (full - 1 - q) / Q + 1 : 0;
        mine = mine_full + (q < halves ? (halves - 1 - q) / Q + 1 : 0);
    }
    struct Item {
        int tm, col0, cols, ncols, which, split, slab0, slabs;   // ncols: accumulator columns
    };
    __device__ Item item(const Params &p, int j) const {
        const int Q = gridDim.x / 2, q = blockIdx.x / 2;
        Item it;
        it.split = it.which = 0;
        int t = q + j * Q, half = -1, tn;
        if (j >= mine_full) {
            const int h = q + (j - mine_full) * Q;
            t = full + h / 2;
            half = h & 1;
        }
        if (p.splits > 1) {
            it.split = t % p.splits;
            t /= p.splits;
        }
        tile_coords(t, p.tiles_m, p.tiles_n, p.group_m, it.tm, tn);
        if (MODE == TWO && tn >= p.out_tiles) {
            it.which = 1;
            tn -= p.out_tiles;
        }
        const int per = MODE == GATE ? p.tile_n / 2 : p.tile_n;   // an output's columns
        it.col0 = tn * per;
        it.cols = per;
        // half a tile where the last wave is cut, or where there are no more columns
        if (half >= 0) it.col0 += half * (per / 2);
        if (half >= 0 || (p.tile_n == TILE && p.N - it.col0 <= per / 2)) it.cols = per / 2;
        it.ncols = MODE == GATE ? 2 * it.cols : it.cols;
        it.slab0 = it.split * p.per_split;
        it.slabs = min(p.per_split, p.slabs - it.slab0);
        return it;
    }
};

template <class T, int PARTS, bool A_MN, bool B_MN, Mode MODE, bool CHUNKS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    pair_gemm_kernel(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB0,
                     const __grid_constant__ CUtensorMap mB1, const Params p, const Output<T> to) {
    constexpr bool SEVERAL = PARTS > 1, BYTES_MODE = MODE == BYTES;
    // the accumulator goes to registers by chunks: of several parts inside the loop over slabs, of
    // one as pieces of the tile with an accumulator each
    constexpr bool CHUNKED = SEVERAL || CHUNKS, PIECES = CHUNKS && !SEVERAL;
    constexpr uint32_t STAGE = 2 * PARTS * PART_BYTES;
    constexpr int STAGES = int(SMEM_RING / STAGE);
    constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(A_MN) << 15) | (uint32_t(B_MN) << 16) |
                               (uint32_t(TILE >> 4) << 24);

    extern __shared__ unsigned char smem_raw[];
    const uintptr_t base = (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023);
    float *stage_out = reinterpret_cast<float *>(base + SMEM_RING);
    uint64_t *full = reinterpret_cast<uint64_t *>(stage_out + EPI_FLOATS);
    uint64_t *empty = full + STAGES;
    uint64_t *acc_full = empty + STAGES;   // [2] MMA -> epilogue (both CTAs)
    uint64_t *acc_empty = acc_full + 2;    // [2] epilogue -> MMA (CTA 0's)
    uint64_t *drain = acc_empty + 2;
    uint32_t *tmem_base = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_base + 1);
    volatile int *issued_slot = abort_flag + 1;

    const uint32_t rank = cluster_ctarank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 2);    // CTA 0's counts one arrival, with bytes, per CTA
            mbar_init(&empty[s], 1);   // the MMA commit, multicast to both CTAs
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], 2 * EPI_WARPS);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        *issued_slot = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc_pair(tmem_base, TMEM_COLUMNS);
    tc_fence_before();
    cluster_barrier();
    tc_fence_after();
    wait_prerequisites();
    launch_dependents();
    const uint32_t taddr = *tmem_base;
    const uint32_t peer_abort = dsmem_map(smem_addr((const void *)abort_flag), rank ^ 1u);
    auto set_abort = [&] {
        *abort_flag = 1;
        st_cluster_flag(peer_abort, 1);
    };

    const int PER_CHUNK = chunk_slabs(SEVERAL, BYTES_MODE) * (BYTES_MODE && to.large && *to.large == 0 ? 2 : 1);
    Work<MODE> work;
    using Item = typename Work<MODE>::Item;
    work.init(p);
    const uint32_t ring = smem_addr(reinterpret_cast<void *>(base));

    if (warp == 0) {
        // ================================================================ copies (both CTAs)
        if (lane == 0) {
            tma_prefetch_desc(&mA);
            tma_prefetch_desc(&mB0);
            tma_prefetch_desc(&mB1);
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            for (int j = 0; j < work.mine && !*abort_flag; ++j) {
                const Item it = work.item(p, j);
                const int arow = it.tm * TILE + int(rank) * ROWS;
                // GATE: the same columns of either matrix; else this CTA's half of the tile's
                const int bcol = it.col0 + (MODE == GATE ? 0 : int(rank) * (it.ncols / 2));
                for (int s = 0; s < it.slabs; ++s) {
                    if (*abort_flag) break;
                    // first use of a stage: parity 1 counts as complete
                    if (!mbar_wait(&empty[stage], phase ^ 1u, p.timeout_ns)) {
                        atomicOr(&g_error_word, ERR_EMPTY_WAIT);
                        set_abort();
                        break;
                    }
                    const uint32_t st = ring + uint32_t(stage) * STAGE;
                    const uint32_t fb = dsmem_map(smem_addr(&full[stage]), 0u);
                    mbar_arrive_expect_tx_cluster(fb, p.slab_bytes);
                    const int slab = SG_IN_RANGE(it.slab0 + s < p.slabs && it.tm < p.tiles_m && stage < STAGES) ? it.slab0 + s : 0;
                    const int second = MODE == SUM && slab >= p.first_slabs ? 1 : 0;
                    const int k = (slab - second * p.first_slabs) * BK;
                    const CUtensorMap *mB = (MODE == GATE ? int(rank) : MODE == SUM ? second : it.which) ? &mB1 : &mB0;
#pragma unroll
                    for (int q = 0; q < PARTS; ++q) {
                        const uint32_t a = st + uint32_t(q) * PART_BYTES, b = a + uint32_t(PARTS) * PART_BYTES;
                        if constexpr (A_MN) {
                            sgp::tma_load_3d_pair(a, &mA, fb, arow, k, q);
                            sgp::tma_load_3d_pair(a + GROUP_BYTES, &mA, fb, arow + 64, k, q);
                        } else {
                            sgp::tma_load_3d_pair(a, &mA, fb, k, arow, second * PARTS + q);
                        }
                        if constexpr (B_MN) {
                            sgp::tma_load_3d_pair(b, mB, fb, bcol, k, q);
                            sgp::tma_load_3d_pair(b + GROUP_BYTES, mB, fb, bcol + 64, k, q);
                        } else {
                            sgp::tma_load_3d_pair(b, mB, fb, k, bcol, q);
                        }
                    }
                    ++issued;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            *issued_slot = issued;
        }
    } else if (warp == 1) {
        // ================================================================ MMA issuer (CTA 0)
        // All lanes go through the loop, what they wait for decided together, and one, elected, issues: in a branch
        // of one lane the operands are not in uniform registers.
        if (rank == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int chunk = 0, piece = 0;   // accumulator hand-overs of several parts; tiles (PIECES: chunks) so far
            bool ok = true;
            auto wait_acc = [&](int a, int use) {   // the epilogues are through with its use - 1
                if (__all_sync(0xffffffffu, mbar_wait_cluster(&acc_empty[a], (uint32_t(use) & 1u) ^ 1u, p.timeout_ns))) {
                    tc_fence_after();
                    return true;
                }
                atomicOr(&g_error_word, ERR_EMPTY_WAIT);
                set_abort();
                return false;
            };
            for (int j = 0; j < work.mine && ok; ++j) {
                const Item it = work.item(p, j);
                const uint32_t idesc = IDESC | (uint32_t(it.ncols >> 3) << 17);
                int begin = 0;
                do {
                    const int end = PIECES ? min(it.slabs, begin + PER_CHUNK) : it.slabs;
                    const int a = SEVERAL ? 0 : piece & 1;
                    // one part: this tile's (or chunk's) accumulator; several: the small pairs'
                    if (!(ok = SEVERAL ? wait_acc(1, piece) : wait_acc(a, piece >> 1))) break;
                    ++piece;
                    for (int s = begin; s < end; ++s) {
                        if (!__all_sync(0xffffffffu, !*abort_flag && mbar_wait_cluster(&full[stage], phase, p.timeout_ns))) {
                            if (!*abort_flag) atomicOr(&g_error_word, ERR_FULL_WAIT);
                            set_abort();
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sa = ring + uint32_t(stage) * STAGE;
                        const uint32_t sb = sa + uint32_t(PARTS) * PART_BYTES;
                        auto mma = [&](uint32_t d, int qa, int qb, int kk, bool accumulate) {
                            sgp::mma_bf16_pair(d, part_desc<A_MN>(sa + uint32_t(qa) * PART_BYTES, kk),
                                               part_desc<B_MN>(sb + uint32_t(qb) * PART_BYTES, kk), idesc, accumulate);
                        };
                        const bool elected = elect_one();
                        if constexpr (SEVERAL) {
                            if (elected)
#pragma unroll
                            for (int kk = 0; kk < BK / 16; ++kk) {
                                bool first = s == 0 && kk == 0;
#pragma unroll
                                for (int qa = PARTS - 1; qa >= 0; --qa)
#pragma unroll
                                    for (int qb = PARTS - 1; qb >= 0; --qb)
                                        if (qa + qb > 0 && qa + qb <= 2) {
                                            mma(taddr + ACC_COLUMNS, qa, qb, kk, !first);
                                            first = false;
                                        }
                            }
                            if (s % PER_CHUNK == 0) {
                                if (!(ok = wait_acc(0, chunk))) break;
                                ++chunk;
                            }
                        }
                        const uint32_t main_acc = taddr + uint32_t(a) * ACC_COLUMNS;
                        if (elected) {
#pragma unroll
                            for (int kk = 0; kk < BK / 16; ++kk)
                                mma(main_acc, 0, 0, kk, SEVERAL ? (s % PER_CHUNK != 0 || kk > 0) : (s > begin || kk > 0));
                            mma_commit_pair(&empty[stage]);   // both CTAs' stage free once read
                            if (SEVERAL && (s % PER_CHUNK == PER_CHUNK - 1 || s == it.slabs - 1)) mma_commit_pair(&acc_full[0]);
                        }
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!SEVERAL && ok && elect_one()) mma_commit_pair(&acc_full[a]);
                    begin = end;
                } while (PIECES && ok && begin < it.slabs);
            }
            if (!ok) {
                // no MMA may still run when either CTA frees its TMEM or exits
                if (elect_one()) mma_commit_pair(drain);
                if (!mbar_wait(drain, 0u, drain_limit_ns(p.timeout_ns)))
                    atomicOr(&g_error_word, ERR_DRAIN_WAIT);
            }
        }
    } else {
        // ================================================================ epilogue (both CTAs)
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t buf = smem_addr(stage_out + (warp - 2) * (32 * (CHUNKED ? 33 : 32)));
        const uint32_t lanes = taddr + (uint32_t(quarter * 32) << 16);
        int turn = 0;
        bool ok = true;
        auto wait_full = [&](int a, int use) {
            if (__any_sync(0xffffffffu, *abort_flag)) return false;
            const bool ready =
                __all_sync(0xffffffffu, mbar_wait(&acc_full[a], uint32_t(use) & 1u, p.timeout_ns));
            if (!ready && lane == 0) {
                atomicOr(&g_error_word, ERR_FULL_WAIT);
                set_abort();
            }
            tc_fence_after();
            return ready;
        };
        auto hand_back = [&](int a) {   // what this warp reads of it is in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(dsmem_map(smem_addr(&acc_empty[a]), 0u));
        };
        for (int j = 0; j < work.mine && ok; ++j) {
            const Item it = work.item(p, j);
            // this warp's columns of an output: 128 or 64, 96 or 32 (GATE: 64, 32)
            const int first_half = (it.cols / 2 + 31) & ~31;
            const int width = half ? it.cols - first_half : first_half;
            const int row0 = it.tm * TILE + int(rank) * ROWS + quarter * 32, rows = min(32, p.M - row0);
            const int col0 = it.col0 + half * first_half;

            // A lane's row of 32 columns from `col`, given two at a time, written a column to a lane; where the sums
            // leave registers for it (64 x 8192 x 4096 bfloat16 weight gradients 82 -> 55 us; beside 128 sums it
            // spilled, and 79 us of float32 became 86) and rows are aligned, four columns to a lane.  SCALED: by the
            // rows' and columns' scales, and the bias (not added where there is none: it would turn -0 into 0).
            const float scale = BYTES_MODE && !p.partial && row0 + lane < p.M ? to.scale[row0 + lane] : 0.0f;   // of this lane's row
            auto write = [&](auto *out, long long ld, int col, auto scaled, auto &&value) {
                using E = std::remove_reference_t<decltype(*out)>;
                constexpr bool SCALED = decltype(scaled)::value;
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 32; i += CHUNKED ? 2 : 4) {
                    const float2 v = value(i);
                    if constexpr (CHUNKED) {
                        sts_float(buf + uint32_t(lane * 33 + i) * 4, v.x);
                        sts_float(buf + uint32_t(lane * 33 + i + 1) * 4, v.y);
                    } else {   // rows 128 bytes apart, their 16-byte pieces swizzled
                        const float2 u = value(i + 2);
                        sts128(buf + uint32_t(lane * 128 + ((i / 4) ^ (lane & 7)) * 16), make_float4(v.x, v.y, u.x, u.y));
                    }
                }
                __syncwarp();
                if (!SG_IN_RANGE(col + 32 <= it.col0 + it.cols && row0 + rows <= (it.tm + 1) * TILE && it.split < p.splits)) return;
                const bool biased = SCALED && to.bias;
                auto finished = [&](float v, float of_row, float of, float bias) {
                    if (!SCALED) return v;
                    v *= of_row * of;
                    return biased ? v + bias : v;
                };
                if constexpr (!CHUNKED) {
                    if (col + 32 <= p.N && ld % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & (4 * sizeof(E) - 1)) == 0) {
                        const int c = col + (lane & 7) * 4, r0 = lane >> 3;
                        float of[4], bias[4];
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            of[d] = SCALED ? to.wscale[c + d] : 0.0f;
                            bias[d] = biased ? sgl::to_f32(to.bias[c + d]) : 0.0f;
                        }
                        E *at = out + (long long)(row0 + r0) * ld + c;
                        // (rows r0, r0 + 8, ... and r0 + 4, r0 + 12, ... have their piece in the same place of the 128 bytes)
                        const uint32_t even = buf + uint32_t(r0 * 128 + ((lane & 7) ^ r0) * 16);
                        const uint32_t odd = buf + uint32_t(r0 * 128 + ((lane & 7) ^ (r0 + 4)) * 16);
#pragma unroll
                        for (int j = 0; j < 8; ++j, at += 4 * ld) {
                            const float of_row = SCALED ? __shfl_sync(0xffffffffu, scale, 4 * j + r0) : 0.0f;
                            const float4 x = lds128((j & 1 ? odd : even) + uint32_t(j * 512));
                            const float v[4] = {finished(x.x, of_row, of[0], bias[0]), finished(x.y, of_row, of[1], bias[1]),
                                                finished(x.z, of_row, of[2], bias[2]), finished(x.w, of_row, of[3], bias[3])};
                            if (4 * j + r0 < rows) sgl::store4(at, v);
                        }
                        return;
                    }
                }
                const int c = col + lane;
                const bool in = c < p.N;
                if (!SCALED && !in) return;
                const float of = SCALED && in ? to.wscale[c] : 0.0f, bias = biased && in ? sgl::to_f32(to.bias[c]) : 0.0f;
                E *at = out + (long long)row0 * ld + c;
                uint32_t from[8];   // of rows 0 to 7, and 8 further on each time
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    from[r] = buf + (CHUNKED ? uint32_t(r * 33 + lane) * 4
                                             : uint32_t(r * 128 + ((lane >> 2) ^ r) * 16 + (lane & 3) * 4));
                for (int r = 0; r < rows; r += 8) {   // (rows: of the whole warp)
#pragma unroll
                    for (int d = 0; d < 8; ++d, at += ld) {
                        const float of_row = SCALED ? __shfl_sync(0xffffffffu, scale, r + d) : 0.0f;
                        const float v = finished(lds32(from[d] + uint32_t(r * (CHUNKED ? 132 : 128))), of_row, of, bias);
                        if (r + d < rows && (!SCALED || in)) *at = sgl::from_f32<E>(v);
                    }
                }
            };
            constexpr std::false_type AS_IT_IS{};
            // 32 columns of the tile's sums: x (and GATE: y, the same columns of U)
            auto finish = [&](int c, const float (&x)[32], const float (&y)[32]) {
                const int col = col0 + c * 32;
                auto xs = [&](int i) { return make_float2(x[i], x[i + 1]); };
                auto ys = [&](int i) { return make_float2(y[i], y[i + 1]); };
                if constexpr (BYTES_MODE) {   // (a range's sums are up to 2^24 here, and stay whole)
                    if (p.partial)
                        write(p.partial + (long long)it.split * p.M * p.N, (long long)p.N, col, AS_IT_IS, [&](int i) {
                            return make_float2(__int_as_float(__float2int_rn(x[i])), __int_as_float(__float2int_rn(x[i + 1])));
                        });
                    else
                        write(to.out, to.ldo, col, std::true_type{}, xs);
                } else if (p.partial) {
                    constexpr int OUTPUTS = MODE == GATE || MODE == TWO ? 2 : 1;
                    const long long ld = (long long)OUTPUTS * p.N;
                    float *out = p.partial + (long long)it.split * p.M * ld + (long long)it.which * p.N;
                    write(out, ld, col, AS_IT_IS, xs);
                    if (MODE == GATE) write(out + p.N, ld, col, AS_IT_IS, ys);
                } else if constexpr (MODE == GATE) {
                    if (to.out) {
                        write(to.out, to.ldo, col, AS_IT_IS, xs);
                        write(to.out1, to.ldo1, col, AS_IT_IS, ys);
                    }
                    sgl::with_act(to.act, [&](auto act) {
                        write(to.H, to.ldh, col, AS_IT_IS, [&](int i) {
                            const float2 v = sgl::gate_value<T, decltype(act)::value>(xs(i));
                            return make_float2(v.x * y[i], v.y * y[i + 1]);
                        });
                    });
                } else {
                    write(it.which ? to.out1 : to.out, it.which ? to.ldo1 : to.ldo, col, AS_IT_IS, xs);
                }
            };

            if constexpr (BYTES_MODE && CHUNKED) {
                int sum[4][32];
                for (int s = 0; s < it.slabs && ok; s += PER_CHUNK, ++turn) {
                    if (!(ok = wait_full(turn & 1, turn >> 1))) break;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (c * 32 >= width) break;
#pragma unroll
                        for (int h = 0; h < 32; h += 16) {
                            float v[16];
                            tmem_add16(lanes + uint32_t(turn & 1) * ACC_COLUMNS + uint32_t(half * first_half + c * 32 + h), v, false);
#pragma unroll
                            for (int i = 0; i < 16; ++i) sum[c][h + i] = __float2int_rn(v[i]) + (s > 0 ? sum[c][h + i] : 0);
                        }
                    }
                    hand_back(turn & 1);
                }
                if (!ok) break;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c * 32 >= width) break;
                    const int col = col0 + c * 32;
                    if (p.partial)   // (they stay whole)
                        write(p.partial + (long long)it.split * p.M * p.N, (long long)p.N, col, AS_IT_IS, [&](int i) {
                            return make_float2(__int_as_float(sum[c][i]), __int_as_float(sum[c][i + 1]));
                        });
                    else
                        write(to.out, to.ldo, col, std::true_type{},
                              [&](int i) { return make_float2(float(sum[c][i]), float(sum[c][i + 1])); });
                }
            } else if constexpr (CHUNKED) {
                float sum[4][32];   // GATE: two of G, two of U
                auto columns = [&](int c) {   // in the accumulator
                    return MODE == GATE ? (c / 2) * it.cols + half * first_half + (c % 2) * 32 : half * first_half + c * 32;
                };
                auto mine = [&](int c) { return (MODE == GATE ? c % 2 : c) * 32 < width; };
                for (int s = 0; s < it.slabs && ok; s += PER_CHUNK, ++turn) {
                    const int a = SEVERAL ? 0 : turn & 1;
                    if (!(ok = wait_full(a, SEVERAL ? turn : turn >> 1))) break;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (mine(c))
#pragma unroll
                            for (int h = 0; h < 32; h += 16)
                                tmem_add16(lanes + uint32_t(a) * ACC_COLUMNS + uint32_t(columns(c) + h), &sum[c][h], s > 0);
                    hand_back(a);
                }
                if (!ok) break;
                if (SEVERAL) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (mine(c))
#pragma unroll
                            for (int h = 0; h < 32; h += 16)
                                tmem_add16(lanes + ACC_COLUMNS + uint32_t(columns(c) + h), &sum[c][h], true);
                    hand_back(1);
                }
#pragma unroll
                for (int c = 0; c < (MODE == GATE ? 2 : 4); ++c)
                    if (c * 32 < width) finish(c, sum[c], sum[MODE == GATE ? c + 2 : c]);
            } else {
                const int a = turn & 1;
                if (!(ok = wait_full(a, turn >> 1))) break;
                ++turn;
#pragma unroll 1
                for (int c = 0; c * 32 < width; ++c) {
                    float x[32], y[32];
                    const uint32_t at = lanes + uint32_t(a) * ACC_COLUMNS + uint32_t(half * first_half + c * 32);
                    tmem_load32(at, x);
                    if (MODE == GATE) tmem_load32(at + uint32_t(it.cols), y);
                    if ((c + 1) * 32 >= width) hand_back(a);
                    finish(c, x, y);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_barrier();   // CTA 0's MMAs and both CTAs' remote arrivals are done
    // After an abort (set in both CTAs before the barrier above), copies may still be
    // landing; only CTA 0 can wait for them: it completes the arrivals of stages that
    // one producer alone filled and waits for the last STAGES fillings.
    if (*abort_flag) {
        if (rank == 0 && threadIdx.x == 0) {
            const int mine = *issued_slot;
            const int peer = ld_cluster_u32(dsmem_map(smem_addr((const void *)issued_slot), 1u));
            const int lo = mine < peer ? mine : peer, hi = mine < peer ? peer : mine;
            for (int q = lo; q < hi; ++q) mbar_arrive(&full[q % STAGES]);
            for (int q = hi > STAGES ? hi - STAGES : 0; q < hi; ++q)
                if (!mbar_wait_cluster(&full[q % STAGES], uint32_t((q / STAGES) & 1),
                                       drain_limit_ns(p.timeout_ns))) {
                    atomicOr(&g_error_word, ERR_DRAIN_WAIT);
                    break;
                }
        }
        cluster_barrier();
    }
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(taddr, TMEM_COLUMNS);
}

}  // namespace sgq
