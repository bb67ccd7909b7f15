// parts_gemm.cuh -- out = A * B on pairs of SMs (tcgen05 `cta_group::2`) where each
// operand is a sum of bfloat16 parts.
//
// A bfloat16 matrix is one part, and so is an 8-bit checkpoint (act8.cuh).  A
// float32 matrix is three: x = x0 + x1 + x2 exactly, each part the leading 8 bits
// of what the ones before leave.  A product of float32 matrices takes the six pairs
// whose parts' ranks add up to at most 2 (what is left out is at most 2^-21 of
// |a||b|, 2^-24 on average); with one part on one side it takes three, and nothing is
// left out.  Six bfloat16 MMAs cost what three TF32 ones do.
//
// The MMA's additions to its fp32 accumulator truncate: sums of n steps come out
// smaller by up to n * 2^-23 (measured: 4.4e-6 of the result at K = 4096 for one
// MMA per 16 k, 2.9e-5 for three per 8).  For float32 the five small pairs have an
// accumulator of their own, which leaves one addition per 16 k in the main one, and every
// CHUNK slabs the main one is added to fp32 registers, round to nearest, and starts over.
// For bfloat16 this happens every LONG_CHUNK slabs.
//
// A 256 x 256 tile to a pair of SMs, 64 k to a slab, persistent; 320 threads:
//   warp 0     copies: each CTA its 128 rows of A and its half of B's columns, by
//              TMA with 128-byte swizzle in either major order, into a ring;
//   warp 1     allocates TMEM; in CTA 0 one thread issues the MMAs;
//   warps 2-9  take the accumulators to registers and write the output.
// One part: two accumulators of 256 columns, the next tile's (or long chunk's) MMAs run under
// this one's epilogue.  Several: main and small, the next chunk's small pairs run while
// the main accumulator is read.
// The rank-side term is more slabs of the same loop: a row's sums stand in the columns
// of its own adapter and zeros in those of the tile's others.  Zero times an adapter's
// value is nothing, unless that is an infinity or a NaN: a tile with such an adapter
// takes the term by FMAs in the epilogue, each row from its own adapter alone.
// Waits are bounded as in tf32x3_pair.cuh, whose abort protocol this is.
//
// Bound by the tensor pipe where the tiles fill whole waves: 8192 x 4096 x 4096 bfloat16 166
// us (1.66 PFLOP/s; the pipe 76 % busy), 4096^3 float32 428 us (1.93 PFLOP/s of bfloat16
// MMAs); at few rows by W's bytes and latency (64 x 4096 x 4096: 18 us with the kernel that
// adds its four ranges).
// 256-column tiles on pairs because a single SM's 128 x 256 would take 96 bytes of operands
// per cycle from L2, a pair's SM takes 64.
#pragma once

#include "kernels.cuh"
#include "parts_gemm.h"
#include "tcgen05.cuh"

namespace sgp {

using namespace sg;
using namespace sg::t3;
using sgl::bf16;

constexpr int TILE = 256, ROWS = 128, BK = 64;
constexpr int EPI_WARPS = 8, THREADS = 64 + 32 * EPI_WARPS;
constexpr uint32_t PART_BYTES = ROWS * BK * 2;              // 16 KB: 128 rows or columns x 64 k
constexpr uint32_t GROUP_BYTES = 64 * BK * 2;               // 8 KB: 64 of them, MN-major
constexpr int EPI_FLOATS = EPI_WARPS * 32 * 33;
constexpr uint32_t TMEM_COLUMNS = 512, ACC_COLUMNS = 256;
constexpr size_t SMEM_RING = 192 * 1024;
constexpr size_t SMEM_BYTES = SMEM_RING + EPI_FLOATS * 4 + 1024 + 256;
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");

struct KernelParams {
    int M, N;
    int tiles_m, tiles_n, group_m;
    int tile_n;             // columns of a tile: 128 to 256, a multiple of 32
    int slabs;              // of 64 k
    int splits, per_split;  // slabs of each range but the last
    const int4 *planes;     // of the rank side, see Product (null: none)
    const int4 *plane_adapter;
    const int *position;
    int most_planes, capacity, width, L;
    float *partial;         // splits x M x N, or null
    unsigned long long timeout_ns;
};

// 3-D tile copy into this CTA's shared memory, counted on a barrier of either CTA.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                                 int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// D (both CTAs' TMEM) = A * B (+ D), bfloat16 operands from both CTAs' shared memory.
__device__ __forceinline__ void mma_bf16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                              bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
        : "memory");
}

// Shared-memory descriptor of a part at k step kk (16 k) of its slab, 128-byte
// swizzle.  K-major: rows of 64 k, 8-row groups 1024 bytes apart, a step is 32
// bytes along the row.  MN-major: rows of 64 rows/columns, one per k, 8-k groups
// 1024 bytes apart and 64-wide groups GROUP_BYTES apart; a step is 16 such rows.
template <bool MN_MAJOR>
__device__ __forceinline__ uint64_t part_desc(uint32_t saddr, int kk) {
    const uint32_t at = saddr + uint32_t(kk) * (MN_MAJOR ? 2048u : 32u);
    return uint64_t((at & 0x3FFFFu) >> 4) | uint64_t(MN_MAJOR ? (GROUP_BYTES >> 4) : 1) << 16 |
           uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 | uint64_t(2) << 61;
}

// The work of pair q of Q: items q, q + Q, ... of `items`: whole tiles, or, with
// `splits` > 1, (tile, range) pairs; without splits a last wave of at most Q / 2
// tiles of 256 columns is cut into half-width tiles.  RANK: (256 rows, four of their planes, range)
// triples, the planes slowest, so that those that hold nothing come last.
template <bool RANK>
struct Items {
    int full, mine_full, mine;

    __device__ void init(const KernelParams &p) {
        const int Q = gridDim.x / 2, q = blockIdx.x / 2;
        const int items = p.tiles_m * p.tiles_n * p.splits, tail = items % Q;
        full = (!RANK && p.tile_n == TILE && p.splits == 1 && tail != 0 && 2 * tail <= Q) ? items - tail : items;
        const int halves = 2 * (items - full);
        mine_full = q < full ? (full - 1 - q) / Q + 1 : 0;
        mine = mine_full + (q < halves ? (halves - 1 - q) / Q + 1 : 0);
    }
    struct Item {
        int tm, col0, ncols, split, slab0, slabs;
        int2 planes;   // the rank side's, of the first range only (RANK: the item's own)
        const int4 *adapters;   // of those planes
    };
    __device__ Item item(const KernelParams &p, int j) const {
        const int Q = gridDim.x / 2, q = blockIdx.x / 2;
        Item it;
        it.split = 0;
        int tn;
        if (j < mine_full) {
            int t = q + j * Q;
            if (p.splits > 1) {
                it.split = t % p.splits;
                t /= p.splits;
            }
            if (RANK)
                it.tm = t % p.tiles_m, tn = t / p.tiles_m;
            else
                tile_coords(t, p.tiles_m, p.tiles_n, p.group_m, it.tm, tn);
            it.col0 = tn * p.tile_n;
            it.ncols = p.N - it.col0 <= TILE / 2 ? TILE / 2 : p.tile_n;
        } else {
            const int h = q + (j - mine_full) * Q;
            tile_coords(full + h / 2, p.tiles_m, p.tiles_n, p.group_m, it.tm, tn);
            it.col0 = tn * TILE + (h & 1) * (TILE / 2);
            it.ncols = TILE / 2;
        }
        it.slab0 = it.split * p.per_split;
        it.slabs = min(p.per_split, p.slabs - it.slab0);
        if (RANK) {
            const int4 all = p.planes[it.tm];
            it.planes = make_int2(all.x + 4 * tn, min(4, all.y - 4 * tn));
            it.adapters = p.plane_adapter + (long long)it.tm * p.most_planes + 4 * tn;
            it.ncols = 64 * it.planes.y;
            if (it.planes.y <= 0) it.slabs = 0;   // nothing here: every role passes it over
        } else {
            const int4 all = p.planes && it.split == 0 ? p.planes[it.tm] : make_int4(0, 0, 1, 0);
            it.planes = make_int2(all.x, all.z ? all.y : -1);
            it.adapters = p.plane_adapter + (long long)it.tm * p.most_planes;
        }
        return it;
    }
};

// Slabs between two visits to the main accumulator of a product of several parts:
// 512 k, 32 truncating additions, 4e-6 at most and a third of that on average.
constexpr int CHUNK = 8;
// The same of one part: 8192 k, 512 additions, 3e-5 of the terms' magnitudes at most (5e-6
// measured), under a hundredth of a bfloat16 spacing.  A kernel of its own (LONG), as the chunks'
// sums in registers cost the shorter products 2 to 3 %: weight gradient of 4096 x 4096 from 16384
// rows 368 us, in one accumulator, whose error grows with the rows (1.1e-4 at 200000), 358; from
// 65536 rows 1440 and 1404.  (16384 rows in chunks of 4096 377, of 2048 382, of 1024 394.)
constexpr int LONG_CHUNK = 128;

// RANK: the rank side's own product, X (256 rows) * [columns of the adapters that the rows
// use, as their planes lie], of which a row keeps its own adapter's columns: sums to
// partial[range][row][width].  LONG: one part, ranges of more than LONG_CHUNK slabs.
template <class T, int PA, int PB, bool A_MN, bool B_MN, bool TRANS, bool RANK, bool LONG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    parts_gemm_kernel(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB,
                      const __grid_constant__ CUtensorMap mH, const __grid_constant__ CUtensorMap mV,
                      const KernelParams p, const Epilogue<T, TRANS> epi) {
    constexpr bool SEVERAL = PA * PB > 1;
    constexpr bool CHUNKED = SEVERAL || RANK || LONG;   // the main accumulator goes to registers by chunks
    constexpr int PER_CHUNK = LONG ? LONG_CHUNK : CHUNK;
    constexpr uint32_t STAGE = (PA + PB) * PART_BYTES;
    constexpr int STAGES = int(SMEM_RING / STAGE);
    constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(A_MN) << 15) |
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

    Items<RANK> items;
    using Item = typename Items<RANK>::Item;
    items.init(p);
    const uint32_t ring = smem_addr(reinterpret_cast<void *>(base));
    // slabs of an item, the rank side's after the product's: with one part a side, the parts of S
    // are planes one after the other
    auto slabs_of = [](const Item &it) {
        return it.slabs + (RANK ? 0 : max(it.planes.y, 0) * (SEVERAL ? 1 : sgl::S_PARTS));
    };

    if (warp == 0) {
        // ================================================================ copies (both CTAs)
        if (lane == 0) {
            tma_prefetch_desc(&mA);
            tma_prefetch_desc(&mB);
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            for (int j = 0; j < items.mine && !*abort_flag; ++j) {
                const Item it = items.item(p, j);
                const int arow = it.tm * TILE + int(rank) * ROWS;
                const int bcol = it.col0 + int(rank) * (it.ncols / 2);
                const int slabs = slabs_of(it);
                for (int s = 0; s < slabs; ++s) {
                    if (*abort_flag) break;
                    // first use of a stage: parity 1 counts as complete
                    if (!mbar_wait(&empty[stage], phase ^ 1u, p.timeout_ns)) {
                        atomicOr(&g_error_word, ERR_EMPTY_WAIT);
                        set_abort();
                        break;
                    }
                    const uint32_t st = ring + uint32_t(stage) * STAGE;
                    const uint32_t fb = dsmem_map(smem_addr(&full[stage]), 0u);
                    mbar_arrive_expect_tx_cluster(
                        fb, RANK ? PA * PART_BYTES + PB * uint32_t(it.ncols / 2) * 128u : STAGE);
                    if (s < it.slabs) {
                        const int k = SG_IN_RANGE(it.slab0 + s < p.slabs && it.tm < p.tiles_m && stage < STAGES)
                                          ? (it.slab0 + s) * BK : 0;
#pragma unroll
                        for (int q = 0; q < PA; ++q) {
                            const uint32_t at = st + uint32_t(q) * PART_BYTES;
                            if constexpr (A_MN) {
                                tma_load_3d_pair(at, &mA, fb, arow, k, q);
                                tma_load_3d_pair(at + GROUP_BYTES, &mA, fb, arow + 64, k, q);
                            } else {
                                tma_load_3d_pair(at, &mA, fb, k, arow, q);
                            }
                        }
                        if constexpr (RANK) {
                            // this CTA's half of the columns, from each adapter at most 32 at a time
                            const int deep = min(p.width, 32);
                            for (int u = 0; u < it.ncols / 2; u += deep) {
                                const int c = int(rank) * (it.ncols / 2) + u, in_plane = c % 64;
                                const int4 of = it.adapters[SG_IN_RANGE(c / 64 < it.planes.y) ? c / 64 : 0];
                                const int slot = p.width < 64 ? in_plane / p.width : 0;
                                const int id = slot == 0 ? of.x : slot == 1 ? of.y : slot == 2 ? of.z : of.w;
                                const int r = p.width < 64 ? in_plane % p.width : of.y + in_plane;
                                const int a = SG_IN_RANGE(id >= 0 && id < p.L && r >= 0 && r + deep <= p.width) ? id : 0;
#pragma unroll
                                for (int q = 0; q < PB; ++q)
                                    tma_load_3d_pair(st + uint32_t(PA + q) * PART_BYTES + uint32_t(u) * 128u, &mB, fb, k,
                                                     r, q * p.L + a);
                            }
                        }
#pragma unroll
                        for (int q = 0; !RANK && q < PB; ++q) {
                            const uint32_t at = st + uint32_t(PA + q) * PART_BYTES;
                            if constexpr (B_MN) {
                                tma_load_3d_pair(at, &mB, fb, bcol, k, q);
                                tma_load_3d_pair(at + GROUP_BYTES, &mB, fb, bcol + 64, k, q);
                            } else {
                                tma_load_3d_pair(at, &mB, fb, k, bcol, q);
                            }
                        }
                    } else if constexpr (!A_MN && !RANK) {
                        const int e = s - it.slabs, part = SEVERAL ? 0 : e / it.planes.y;
                        const int in_tile = SEVERAL ? e : e % it.planes.y;
                        const int plane = SG_IN_RANGE(in_tile < p.most_planes && part < sgl::S_PARTS && it.planes.x >= 0 &&
                                                      it.planes.x + in_tile < p.capacity) ? it.planes.x + in_tile : 0;
#pragma unroll
                        for (int q = 0; q < PA; ++q)
                            tma_load_3d_pair(st + uint32_t(q) * PART_BYTES, &mH, fb, 0, int(rank) * ROWS,
                                             (part + q) * p.capacity + plane);
                        const int4 of = it.adapters[in_tile];
                        const int deep = min(p.width, BK);   // rank columns of an adapter in this plane
#pragma unroll
                        for (int q = 0; q < PB; ++q)
                            for (int u = 0; u * deep < BK; ++u) {
                                const uint32_t at =
                                    st + uint32_t(PA + q) * PART_BYTES + uint32_t(u * deep) * 128u;
                                const int id = u == 0 ? of.x : u == 1 ? of.y : u == 2 ? of.z : of.w;
                                const int r = deep == BK ? of.y : 0;
                                const int a = SG_IN_RANGE(id >= 0 && id < p.L && r >= 0 && r + deep <= p.width) ? id : 0;
                                tma_load_3d_pair(at, &mV, fb, bcol, r, q * p.L + a);
                                tma_load_3d_pair(at + GROUP_BYTES, &mV, fb, bcol + 64, r, q * p.L + a);
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
        if (lane == 0 && rank == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int chunk = 0, tile = 0;   // accumulator hand-overs, tiles (LONG: chunks) so far
            bool ok = true;
            auto wait_acc = [&](int a, int use) {   // the epilogues are through with its use - 1
                if (mbar_wait_cluster(&acc_empty[a], (uint32_t(use) & 1u) ^ 1u, p.timeout_ns)) {
                    tc_fence_after();
                    return true;
                }
                atomicOr(&g_error_word, ERR_EMPTY_WAIT);
                set_abort();
                return false;
            };
            for (int j = 0; j < items.mine && ok; ++j) {
                const Item it = items.item(p, j);
                const uint32_t idesc = IDESC | (uint32_t(it.ncols >> 3) << 17);
                const int slabs = slabs_of(it);
                if (RANK && slabs == 0) continue;
                // Several parts and RANK: chunks begin and end inside the loop over slabs.  (So they
                // could here, but that made a slab of one MMA per 16 k 11 % longer.)
                constexpr bool INSIDE = SEVERAL || RANK;
                int begin = 0;
                do {
                    const int end = LONG ? min(slabs, begin + LONG_CHUNK) : slabs;
                    const int a = INSIDE ? 0 : tile & 1;
                    int main_buf = a;
                    // one part: this tile's (LONG: chunk's) accumulator; several: the small pairs'
                    if (SEVERAL && !(ok = wait_acc(1, tile))) break;
                    if (!INSIDE && !(ok = wait_acc(a, tile >> 1))) break;
                    ++tile;
                    for (int s = begin; s < end; ++s) {
                        if (*abort_flag || !mbar_wait_cluster(&full[stage], phase, p.timeout_ns)) {
                            if (!*abort_flag) atomicOr(&g_error_word, ERR_FULL_WAIT);
                            set_abort();
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sa = ring + uint32_t(stage) * STAGE;
                        const uint32_t sb = sa + uint32_t(PA) * PART_BYTES;
                        const bool rank_side = s >= it.slabs;   // (its stack is MN-major)
                        auto mma = [&](uint32_t d, int qa, int qb, int kk, bool accumulate) {
                            const uint32_t b = sb + uint32_t(qb) * PART_BYTES;
                            const bool mn = B_MN || rank_side;
                            mma_bf16_pair(d, part_desc<A_MN>(sa + uint32_t(qa) * PART_BYTES, kk),
                                          mn ? part_desc<true>(b, kk) : part_desc<false>(b, kk),
                                          idesc | (uint32_t(mn) << 16), accumulate);
                        };
                        if constexpr (SEVERAL) {
                            const uint32_t small = taddr + ACC_COLUMNS;
#pragma unroll
                            for (int kk = 0; kk < BK / 16; ++kk) {
                                bool first = s == 0 && kk == 0;
#pragma unroll
                                for (int qa = PA - 1; qa >= 0; --qa)
#pragma unroll
                                    for (int qb = PB - 1; qb >= 0; --qb)
                                        if (qa + qb > 0 && qa + qb <= 2) {
                                            mma(small, qa, qb, kk, !first);
                                            first = false;
                                        }
                            }
                        }
                        // (one part leaves TMEM for two main accumulators, taken in turn)
                        if (INSIDE && s % PER_CHUNK == 0) {
                            main_buf = SEVERAL ? 0 : chunk & 1;
                            if (!(ok = wait_acc(main_buf, SEVERAL ? chunk : chunk >> 1))) break;
                            ++chunk;
                        }
                        const uint32_t main_acc = taddr + uint32_t(main_buf) * ACC_COLUMNS;
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            mma(main_acc, 0, 0, kk, INSIDE ? (s % PER_CHUNK != 0 || kk > 0) : (s > begin || kk > 0));
                        mma_commit_pair(&empty[stage]);   // both CTAs' stage free once read
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                        if (INSIDE && (s % PER_CHUNK == PER_CHUNK - 1 || s == slabs - 1))
                            mma_commit_pair(&acc_full[main_buf]);
                    }
                    if (!INSIDE && ok) mma_commit_pair(&acc_full[a]);
                    begin = end;
                } while (LONG && ok && begin < slabs);
            }
            if (!ok) {
                // no MMA may still run when either CTA frees its TMEM or exits
                mma_commit_pair(drain);
                if (!mbar_wait(drain, 0u, drain_limit_ns(p.timeout_ns)))
                    atomicOr(&g_error_word, ERR_DRAIN_WAIT);
            }
        }
    } else {
        // ================================================================ epilogue (both CTAs)
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        float *buf = stage_out + (warp - 2) * (32 * 33);
        const uint32_t lanes = uint32_t(quarter * 32) << 16;
        int chunk = 0, done = 0;
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
        for (int j = 0; j < items.mine && ok; ++j) {
            const Item it = items.item(p, j);
            if (RANK && it.slabs == 0) continue;
            const int first_half = (it.ncols / 2 + 31) & ~31;   // this warp's columns: 128, 96, 64 or 32
            const int width = half ? it.ncols - first_half : first_half;
            const int row0 = it.tm * TILE + int(rank) * ROWS + quarter * 32;
            const int col0 = it.col0 + half * first_half;
            const bool fma_expand = it.planes.y < 0 && p.partial == nullptr;

            auto write = [&](int c, const float (&v)[32]) {   // columns col0 + 32 c ..
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 32; ++i) buf[lane * 33 + i] = v[i];
                __syncwarp();
                const int col = col0 + c * 32 + lane;
                if (col >= p.N) return;
                const int rows = min(32, p.M - row0);
                if (!SG_IN_RANGE(col < it.col0 + it.ncols && row0 + rows <= (it.tm + 1) * TILE && it.split < p.splits)) return;
                if (p.partial) {
                    float *out = p.partial + ((long long)it.split * p.M + row0) * p.N + col;
                    for (int r = 0; r < rows; ++r) out[(long long)r * p.N] = buf[r * 33 + lane];
                    return;
                }
                const float bias = epi.bias ? sgl::to_f32(epi.bias[col]) : 0.0f;
                T *out = epi.out + (long long)row0 * epi.ldo + col;
                if (!fma_expand && epi.beta == 0.0f) {
#pragma unroll 8
                    for (int r = 0; r < rows; ++r)
                        out[(long long)r * epi.ldo] = sgl::from_f32<T>(buf[r * 33 + lane] + bias);
                    return;
                }
                for (int r = 0; r < rows; ++r) {
                    float x = buf[r * 33 + lane] + bias;
                    const int a = fma_expand ? epi.ad.of_row(row0 + r) : -1;
                    if (a >= 0) {
                        const int n = epi.ad.rank(a);
                        const float *S = epi.S + (row0 + r) * epi.lds;
                        const T *V = epi.V.matrix(a) + (TRANS ? col * epi.V.ld : col);
#pragma unroll 4
                        for (int k = 0; k < n; ++k)
                            x = fmaf(S[k], sgl::to_f32(V[TRANS ? k : k * epi.V.ld]), x);
                    }
                    if (epi.beta != 0.0f) x = fmaf(epi.beta, sgl::to_f32(out[(long long)r * epi.ldo]), x);
                    out[(long long)r * epi.ldo] = sgl::from_f32<T>(x);
                }
            };

            if constexpr (CHUNKED) {
                const int slabs = slabs_of(it);
                float sum[4][32];
                for (int s = 0; s < slabs && ok; s += PER_CHUNK, ++chunk) {
                    const int buf = SEVERAL ? 0 : chunk & 1;
                    if (!(ok = wait_full(buf, SEVERAL ? chunk : chunk >> 1))) break;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (c * 32 >= width) break;
#pragma unroll
                        for (int h = 0; h < 32; h += 16)
                            tmem_add16(taddr + uint32_t(buf) * ACC_COLUMNS + lanes + uint32_t(half * first_half + c * 32 + h),
                                       &sum[c][h], s > 0);
                    }
                    hand_back(buf);
                }
                if (!ok) break;
#pragma unroll
                for (int c = 0; SEVERAL && c < 4; ++c) {
                    if (c * 32 >= width) break;
#pragma unroll
                    for (int h = 0; h < 32; h += 16)
                        tmem_add16(taddr + ACC_COLUMNS + lanes + uint32_t(half * first_half + c * 32 + h), &sum[c][h],
                                   true);
                }
                if (SEVERAL) hand_back(1);
                if constexpr (RANK) {   // a lane has a row's columns: it keeps its adapter's
                    const int row = row0 + lane, of = row < p.M ? epi.ad.of_row(row) : -1;
                    const bool any = of >= 0 && epi.ad.rank(of) > 0;
                    const int first = any ? p.position[row] * p.width : 0;
                    float *out = p.partial + ((long long)it.split * p.M + row) * p.width;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const int r = col0 + c * 32 + i - first;   // a multiple of 4, as all of these are
                            if (any && c * 32 < width && r >= 0 && r < p.width && SG_IN_RANGE(it.split < p.splits && r + 4 <= p.width))
                                *reinterpret_cast<float4 *>(out + r) =
                                    make_float4(sum[c][i], sum[c][i + 1], sum[c][i + 2], sum[c][i + 3]);
                        }
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c * 32 < width) write(c, sum[c]);
                }
            } else {
                const int a = done & 1;
                if (!(ok = wait_full(a, done >> 1))) break;
                ++done;
#pragma unroll 1
                for (int c = 0; c * 32 < width; ++c) {
                    float v[32];
                    tmem_load32(taddr + uint32_t(a) * ACC_COLUMNS + lanes + uint32_t(half * first_half + c * 32), v);
                    if ((c + 1) * 32 >= width) hand_back(a);
                    write(c, v);
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

// The ranges' partial sums added in order, and the epilogue; a thread to an element.
template <class T, bool TRANS>
__global__ void __launch_bounds__(256)
    finish_kernel(int M, int N, int splits, const float *__restrict__ partial, const int4 *planes, int row0,
                  Epilogue<T, TRANS> epi) {
    const long long i = blockIdx.y;
    const int j = blockIdx.x * 256 + threadIdx.x;
    if (j >= N || !SG_IN_RANGE(row0 + i < M)) return;
    wait_prerequisites();
    launch_dependents();
    float x = epi.bias ? sgl::to_f32(epi.bias[j]) : 0.0f;
    const long long plane = (long long)M * N;
    float sum = 0.0f;
#pragma unroll 8
    for (int s = 0; s < splits; ++s) sum += partial[s * plane + i * N + j];
    x += sum;
    const int a = planes && planes[(row0 + i) / TILE].z ? -1 : epi.ad.of_row(i);
    if (a >= 0) {
        const int n = epi.ad.rank(a);
        const float *S = epi.S + i * epi.lds;
        const T *V = epi.V.matrix(a) + (TRANS ? j * epi.V.ld : j);
#pragma unroll 8
        for (int k = 0; k < n; ++k) x = fmaf(S[k], sgl::to_f32(V[TRANS ? k : k * epi.V.ld]), x);
    }
    T *out = epi.out + i * epi.ldo + j;
    if (epi.beta != 0.0f) x = fmaf(epi.beta, sgl::to_f32(*out), x);
    *out = sgl::from_f32<T>(x);
}

}  // namespace sgp
