// byte_tiles.cuh -- the product of int8 matrices of up to 256 rows to a tile on the tensor cores, W brought
// to float16 on its way into shared memory.
//
// Bound by reading W once.  The rows are the MMA's narrow side: a tile is 128 columns of W (the MMA's M) by
// up to 256 rows of X (its N), and a block has one tile and one range of at most 1024 of the
// contraction.  Every int8 is exactly a float16, a sum of 1024 products of two is at most 2^24, so
// the fp32 accumulator holds it exactly; the ranges' sums are added as int32 (byte_finish_kernel).
//
// 288 threads.  Warps 0 to 7 copy 64 k at a time, several slabs ahead (16 bytes to a copy, each
// thread its own bytes in its own slots, so that a copy is waited for without a barrier), turn
// their bytes into float16 (a byte plus 128 under the exponent of 1024, less 1152: three
// instructions for four) and store them where the MMA wants them (128-byte swizzle: W with its
// columns, X with its k next to each other).  Warp 8 issues the MMAs.  At the end warps 0 to 7 take the
// accumulator out, a lane to a column of W.
//
// W's rows that are not 16-byte aligned take two copies, and their bytes are shifted into place in
// registers.
#pragma once

#include "linear8.cuh"
#include "parts_gemm.cuh"

namespace sgl {

constexpr int TILE_COLS = 128, TILE_K = 64, TILE_RANGE = 1024, TILE_THREADS = 288, TILE_COPIERS = 256;

struct TileWork {
    int M, N, K;
    int across, down, ranges, range;   // tiles of columns, of rows; range: a multiple of 64
    int rows;                          // of a tile: a multiple of 16
    int *partial;                      // ranges x M x N; null (one range): Y
    unsigned long long timeout_ns;
};

// ROWS: of a tile at most.  ALIGNED: the rows of W and of q can be copied 16 bytes at a time.
template <int ROWS, bool ALIGNED>
struct ByteTile {
    static constexpr int BLOCKS = ROWS <= 64 ? 2 : 1;          // to an SM
    static constexpr int W_UNITS = 2, X_UNITS = ROWS * 4 > TILE_COPIERS ? ROWS * 4 / TILE_COPIERS : 1;   // of 16 bytes, to a thread
    static constexpr int UNIT = ALIGNED ? 1 : 2;               // copies to a unit
    static constexpr int SLAB = (W_UNITS + X_UNITS) * UNIT * 16 * TILE_COPIERS;
    static constexpr int DEPTH = ROWS == 256 && !ALIGNED ? 2 : ROWS == 128 && ALIGNED ? 6 : ALIGNED ? 4 : ROWS <= 64 ? 2 : 3;
    static constexpr int W_BYTES = TILE_COLS * TILE_K * 2, X_BYTES = ROWS * TILE_K * 2, STAGE = W_BYTES + X_BYTES, STAGES = 2;
    static constexpr size_t SMEM = size_t(STAGES) * STAGE + size_t(DEPTH) * SLAB + 1024 + 128;
    static constexpr uint32_t TMEM = ROWS < 32 ? 32 : ROWS;
    static_assert(SMEM * BLOCKS + 1024 * BLOCKS <= 228 * 1024, "shared memory of an SM");
};

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
        : "memory");
}

// Four int8 as two words of float16.
__device__ __forceinline__ uint2 halves_of(uint32_t w) {
    w ^= 0x80808080u;
    const uint32_t lo = __byte_perm(w, 0x64646464u, 0x4140), hi = __byte_perm(w, 0x64646464u, 0x4342);
    uint2 out;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(out.x) : "r"(lo), "r"(0x64806480u));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(out.y) : "r"(hi), "r"(0x64806480u));
    return out;
}

// Bytes from `shift` of the 32 in a and b.
__device__ __forceinline__ uint4 shifted(uint4 a, uint4 b, int shift) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (shift & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (shift & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const int bits = (shift & 3) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

template <class T, int ROWS, bool ALIGNED>
__global__ void __launch_bounds__(TILE_THREADS, ByteTile<ROWS, ALIGNED>::BLOCKS)
    byte_tiles_kernel(const TileWork w, const signed char *X, long long ldx, const signed char *W, long long ldw,
                      const float *scale, const float *wscale, const T *bias, T *Y, long long ldy) {
    using Z = ByteTile<ROWS, ALIGNED>;
    using namespace sg;
    using namespace sg::t3;
    extern __shared__ unsigned char smem_tiles[];
    const uintptr_t base = (reinterpret_cast<uintptr_t>(smem_tiles) + 1023) & ~uintptr_t(1023);
    const uint32_t stages = smem_addr(reinterpret_cast<void *>(base)), raw = stages + Z::STAGES * Z::STAGE;
    uint64_t *full = reinterpret_cast<uint64_t *>(base + Z::STAGES * Z::STAGE + Z::DEPTH * Z::SLAB);
    uint64_t *empty = full + Z::STAGES;
    uint64_t *done = empty + Z::STAGES;
    uint32_t *tmem_base = reinterpret_cast<uint32_t *>(done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_base + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < Z::STAGES; ++s) {
            mbar_init(&full[s], TILE_COPIERS / 32);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == TILE_COPIERS / 32) tmem_alloc(tmem_base, Z::TMEM);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wait_prerequisites();
    launch_dependents();
    const uint32_t taddr = *tmem_base;

    // blocks of the same columns and range are neighbours: their W comes from L2
    int b = int(blockIdx.x);
    const int tm = b % w.down;
    b /= w.down;
    const int n0 = (b % w.across) * TILE_COLS, q = b / w.across;
    const int m0 = tm * w.rows, rows = min(w.rows, (w.M - m0 + 15) & ~15);   // of the MMA
    const int k0 = q * w.range, kn = min(w.range, w.K - k0), slabs = (kn + TILE_K - 1) / TILE_K;
    const bool sane = SG_IN_RANGE(kn > 0 && kn <= TILE_RANGE && n0 < w.N && m0 < w.M && q < w.ranges && rows <= ROWS);

    bool ok = sane;
    auto give_up = [&](unsigned what) {
        atomicOr(&g_error_word, what);
        *abort_flag = 1;
        ok = false;
    };
    if (warp < TILE_COPIERS / 32) {
        // ================================================================ copies and conversion
        const int t = threadIdx.x;
        // Unit i of W: 16 columns of row k of the slab; of X: 16 k of a row.
        auto w_at = [&](int i, int &k, int &c) { k = (t + i * TILE_COPIERS) >> 3, c = (t & 7) * 16; };
        auto x_at = [&](int i, int &m, int &k) { m = (t + i * TILE_COPIERS) >> 2, k = (t & 3) * 16; };
        auto slot = [&](int depth, int unit, int part) {
            return raw + uint32_t(depth * Z::SLAB + ((unit * Z::UNIT + part) * TILE_COPIERS + t) * 16);
        };
        // `n` bytes from p (at most 16, the rest zero; `first`: the matrix's first byte) to a unit's slots.
        auto copy = [&](int depth, int unit, const signed char *p, int n, const signed char *first) {
            n = max(0, min(16, n));
            if constexpr (ALIGNED) {
                cp_async16(slot(depth, unit, 0), n > 0 ? p : first, uint32_t(n));
            } else {
                const int shift = int(reinterpret_cast<uintptr_t>(p) & 15);
                const signed char *from = p - shift;
                if (from < first && n > 0) {   // (it would begin before the matrix)
                    uint32_t word[8] = {};
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (i < n) {
                            const int at = shift + i;
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (at >> 2 == j) word[j] |= (uint32_t(p[i]) & 0xffu) << (8 * (at & 3));
                        }
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(slot(depth, unit, 0)), "r"(word[0]),
                                 "r"(word[1]), "r"(word[2]), "r"(word[3]) : "memory");
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(slot(depth, unit, 1)), "r"(word[4]),
                                 "r"(word[5]), "r"(word[6]), "r"(word[7]) : "memory");
                } else {
                    const int head = n > 0 ? min(16, shift + n) : 0, tail = n > 0 ? max(0, shift + n - 16) : 0;
                    const signed char *some = reinterpret_cast<const signed char *>(reinterpret_cast<uintptr_t>(first) & ~uintptr_t(15));
                    cp_async16(slot(depth, unit, 0), head ? from : some, uint32_t(head));
                    cp_async16(slot(depth, unit, 1), tail ? from + 16 : some, uint32_t(tail));
                }
            }
        };
        auto issue = [&](int s) {
            if (s < slabs) {
                const int depth = s % Z::DEPTH, ks = s * TILE_K;
#pragma unroll
                for (int i = 0; i < Z::W_UNITS; ++i) {
                    int k, c;
                    w_at(i, k, c);
                    copy(depth, i, W + (long long)(k0 + ks + k) * ldw + n0 + c, ks + k < kn ? w.N - n0 - c : 0, W);
                }
#pragma unroll
                for (int i = 0; i < Z::X_UNITS; ++i) {
                    int m, k;
                    x_at(i, m, k);
                    if (m < ROWS)
                        copy(depth, Z::W_UNITS + i, X + (long long)(m0 + m) * ldx + k0 + ks + k,
                             m < rows && m0 + m < w.M ? kn - ks - k : 0, X);
                }
            }
            cp_async_commit();
        };
        auto take = [&](int depth, int unit, const signed char *p) {
            auto load = [&](int part) {
                uint4 v;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(slot(depth, unit, part)) : "memory");
                return v;
            };
            if constexpr (ALIGNED) return load(0);
            return shifted(load(0), load(1), int(reinterpret_cast<uintptr_t>(p) & 15));
        };
        // 16 values to the halves of a 128-byte line: chunks `chunk` and the one after, swizzled
        auto put = [&](uint32_t line, int chunk, int row, uint4 v) {
            const uint2 a = halves_of(v.x), b = halves_of(v.y), c = halves_of(v.z), d = halves_of(v.w);
            const uint32_t at = line + uint32_t((chunk ^ (row & 7)) << 4), at1 = line + uint32_t(((chunk + 1) ^ (row & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a.x), "r"(a.y), "r"(b.x), "r"(b.y) : "memory");
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at1), "r"(c.x), "r"(c.y), "r"(d.x), "r"(d.y) : "memory");
        };
        if (sane) {
#pragma unroll 1
            for (int s = 0; s < Z::DEPTH; ++s) issue(s);
        }
        uint32_t phase = 0;
        for (int s = 0; s < slabs && ok; ++s) {
            const int stage = s % Z::STAGES, depth = s % Z::DEPTH, ks = s * TILE_K;
            cp_async_wait<Z::DEPTH - 1>();
            // first use of a stage: parity 1 counts as complete
            if (*abort_flag || !mbar_wait(&empty[stage], phase ^ 1u, w.timeout_ns)) {
                if (!*abort_flag) atomicOr(&g_error_word, ERR_EMPTY_WAIT);
                *abort_flag = 1;
                ok = false;
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t st = stages + uint32_t(stage * Z::STAGE);
#pragma unroll
            for (int i = 0; i < Z::W_UNITS; ++i) {
                int k, c;
                w_at(i, k, c);
                put(st + uint32_t((c >> 6) * sgp::GROUP_BYTES + k * 128), (c & 63) >> 3, k,
                    take(depth, i, W + (long long)(k0 + ks + k) * ldw + n0 + c));
            }
#pragma unroll
            for (int i = 0; i < Z::X_UNITS; ++i) {
                int m, k;
                x_at(i, m, k);
                if (m < rows)
                    put(st + uint32_t(Z::W_BYTES + m * 128), k >> 3, m,
                        take(depth, Z::W_UNITS + i, X + (long long)(m0 + m) * ldx + k0 + ks + k));
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the MMA reads them
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[stage]);
            issue(s + Z::DEPTH);
            if (stage == Z::STAGES - 1) phase ^= 1u;
        }
        cp_async_wait<0>();
    } else if (lane == 0) {
        // ================================================================ MMA issuer
        const uint32_t idesc = (1u << 4) | (1u << 15) | (uint32_t(rows >> 3) << 17) | (uint32_t(TILE_COLS >> 4) << 24);
        uint32_t phase = 0;
        for (int s = 0; s < slabs && ok; ++s) {
            const int stage = s % Z::STAGES;
            if (*abort_flag || !mbar_wait(&full[stage], phase, w.timeout_ns)) {
                give_up(*abort_flag ? 0u : ERR_FULL_WAIT);
                break;
            }
            tc_fence_after();
            const uint32_t st = stages + uint32_t(stage * Z::STAGE);
#pragma unroll
            for (int kk = 0; kk < TILE_K / 16; ++kk)
                mma_f16(taddr, sgp::part_desc<true>(st, kk), sgp::part_desc<false>(st + Z::W_BYTES, kk), idesc, s > 0 || kk > 0);
            mma_commit(&empty[stage]);
            if (stage == Z::STAGES - 1) phase ^= 1u;
        }
        mma_commit(done);   // of all that were issued
        if (!mbar_wait(done, 0u, drain_limit_ns(w.timeout_ns))) give_up(ERR_DRAIN_WAIT);
    }
    __syncthreads();
    if (sane && !*abort_flag && warp < TILE_COPIERS / 32) {
        // ================================================================ the sums, a lane to a column
        tc_fence_after();
        const int quarter = warp & 3, col = n0 + quarter * 32 + lane;
        const float of = !w.partial && col < w.N ? wscale[col] : 0.0f;
        const float add = !w.partial && bias && col < w.N ? to_f32(bias[col]) : 0.0f;
        for (int c = (warp >> 2) * 16; c < rows; c += 32) {
            float v[16];
            tmem_add16(taddr + (uint32_t(quarter * 32) << 16) + uint32_t(c), v, false);
            if (col >= w.N) continue;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const long long m = m0 + c + i;
                if (m >= w.M || c + i >= rows) continue;
                if (w.partial) {
                    w.partial[((long long)q * w.M + m) * w.N + col] = __float2int_rn(v[i]);
                } else {
                    const float y = v[i] * (scale[m] * of);
                    Y[m * ldy + col] = from_f32<T>(bias ? y + add : y);
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == TILE_COPIERS / 32) {
        __syncwarp();
        tmem_dealloc(taddr, Z::TMEM);
    }
}

}  // namespace sgl
