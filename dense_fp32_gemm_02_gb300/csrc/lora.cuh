// lora.cuh -- kernels of the adapter layer and of the weight gradient from a
// checkpoint.
#pragma once

#include "act8.cuh"
#include "adapters.cuh"
#include "kernels.cuh"

namespace sgl {

// A matrix read as fp32 elements: a row-major array, or a checkpoint.
template <class T>
struct Rows {
    const T *p;
    long long ld;
    __device__ float at(long long i, long long j) const { return to_f32(p[i * ld + j]); }
    __device__ void at8(long long i, long long j, float (&v)[8]) const { load8(p + i * ld + j, v); }
};
struct Act8Rows {
    const signed char *q, *e;
    long long ldq, lde;
    __device__ float at(long long i, long long j) const {
        return float(q[i * ldq + j]) * act8_step(e[i * lde + j / ACT8_BLOCK]);
    }
    __device__ void at8(long long i, long long j, float (&v)[8]) const {   // within a block
        const uint2 w = *reinterpret_cast<const uint2 *>(q + i * ldq + j);
        const float step = act8_step(e[i * lde + j / ACT8_BLOCK]);
        unpack_s8(w.x, v);
        unpack_s8(w.y, v + 4);
#pragma unroll
        for (int d = 0; d < 8; ++d) v[d] *= step;
    }
};

// ------------------------------------------------------------------ parts
// x as a sum of up to three bfloat16, each the leading 8 bits of what the ones before
// leave (cut, not rounded: x = x0 + x1 + x2 exactly, and no part overflows; below 2^-110 what
// lies under 2^-133, the least bfloat16, is lost).  What is
// not finite stays in the last, which a product of parts takes with the other side's first alone:
// infinity times a part that is zero only because the number has few bits would be NaN.  (The
// first is then 1 of its sign, for infinity times infinity.)
__device__ __forceinline__ void split_parts(float x, float (&part)[3]) {
    const float head = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
    float rest = x - head;
    const bool finite = fabsf(rest) < 3.0e38f;   // not for an infinity or a NaN
    rest = finite ? rest : 0.0f;
    part[0] = finite ? head : copysignf(1.0f, x);
    part[1] = __uint_as_float(__float_as_uint(rest) & 0xffff0000u);
    part[2] = finite ? rest - part[1] : x + x;   // (x + x: a NaN whose leading bits say so)
}

// Two floats that are bfloat16 already as a word (the first in the low half).
__device__ __forceinline__ uint32_t pack_exact(float lo, float hi) {
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}

// Where the parts of a matrix go: `planes` apart, rows `pitch` apart (both multiples
// of 8 elements, 16-byte aligned).
struct Parts {
    bf16 *p;
    long long pitch, plane;
};

// Eight consecutive elements of a row as PARTS planes.
template <int PARTS>
__device__ __forceinline__ void store_parts(const Parts &to, long long row, long long col,
                                            const float (&x)[8]) {
    float part[8][3];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (PARTS == 1) {
            part[i][0] = x[i];
        } else {
            split_parts(x[i], part[i]);
        }
    }
    bf16 *at = to.p + row * to.pitch + col;
#pragma unroll
    for (int q = 0; q < PARTS; ++q)
        *reinterpret_cast<uint4 *>(at + q * to.plane) =
            make_uint4(pack_exact(part[0][q], part[1][q]), pack_exact(part[2][q], part[3][q]),
                       pack_exact(part[4][q], part[5][q]), pack_exact(part[6][q], part[7][q]));
}

// A matrix and where its parts go.  `wide`: its rows are 16-byte aligned (8-byte for a
// checkpoint's q).  No rows: nothing to do.
template <class X>
struct PartsJob {
    X x;
    int rows, cols;
    bool wide;
    Parts to;
    Divisor per_row;     // octets

    PartsJob(X x_, int rows_, int cols_, bool wide_, Parts to_)
        : x(x_), rows(rows_), cols(cols_), wide(wide_), to(to_),
          per_row(Divisor::of(cols > 0 ? unsigned((cols + 7LL) / 8) : 1u)) {}
    __host__ __device__ long long octets() const { return (long long)rows * ((cols + 7LL) / 8); }
};

// Octets t, t + step, ... of a job: a thread to eight columns of a row.
template <int PARTS, class X>
__device__ __forceinline__ void take_parts(const PartsJob<X> &job, long long t, long long step) {
    const long long total = job.octets();
    const bool small = total <= 0x7fffffffll;
    for (; t < total; t += step) {
        const long long i = small ? (long long)job.per_row.quotient(unsigned(t)) : t / job.per_row.d;
        const int c = int(t - i * job.per_row.d) * 8;
        if (!SG_IN_RANGE(i >= 0 && i < job.rows && c >= 0 && c < job.cols && c + 8 <= job.to.pitch &&
                         (i + 1) * job.to.pitch <= job.to.plane))
            continue;
        float v[8];
        if (job.wide && c + 8 <= job.cols) {
            job.x.at8(i, c, v);
        } else {
#pragma unroll
            for (int d = 0; d < 8; ++d) v[d] = c + d < job.cols ? job.x.at(i, c + d) : 0.0f;
        }
        store_parts<PARTS>(job.to, i, c, v);
    }
}

// The parts of the product's operands that the TMA cannot read in place.  `beside`: the
// kernel before it groups the rows, and need only have ended when this one ends (host_state.h).
template <int P_PARTS, int Q_PARTS, class XP, class XQ>
__global__ void __launch_bounds__(256) parts_kernel(PartsJob<XP> p, PartsJob<XQ> q, bool beside) {
    if (!beside) sg::wait_prerequisites();
    sg::launch_dependents();
    const long long t = (long long)blockIdx.x * 256 + threadIdx.x, step = (long long)gridDim.x * 256;
    take_parts<P_PARTS>(p, t, step);
    take_parts<Q_PARTS>(q, t, step);
    if (beside && blockIdx.x == 0) sg::wait_prerequisites();
}

// ------------------------------------------------------------------ rows by adapter
// Rows grouped by their adapter, in the order of the rows within a group (a stable
// counting sort), and the work list of the kernel that walks the groups.  Rows
// without an adapter, or with one of rank 0, come last, as group L.
//
// For the tensor cores, each 256 rows (a tile of the product) also get their rank-side
// operand laid out: the adapters that occur in the tile, in ascending order, take `width`
// columns each, and 64 columns make a plane of 256 x 64, in which a row has its own sums
// in its own adapter's columns and zeros elsewhere.
struct Groups {
    int *perm;           // M: row numbers, group after group
    int4 *chunks;        // of up to `chunk` rows of an adapter: {adapter, first place in perm,
                         // rows, 0}, max_chunks of them, the last without rows
    int *chunk_begin;    // L + 1: the chunks of adapter a are [a], .. [a + 1]
    int max_chunks, chunk;
    int *used;           // L: whether a row uses the adapter
    int *unclean;        // L: whether it holds something that is not finite (pack_stack)
    int4 *planes;        // for each 256 rows {first plane, planes, 1 if the product may use them
                         // (not past the capacity, nor with an unclean adapter), 0}
    int4 *plane_adapter; // most_planes for each 256 rows: a plane's 64 / width adapters (the
                         // last one repeated), or {adapter, first rank column} where width >= 64
    int *position;       // M: which of its tile's adapters a row uses
    int most_planes;     // of 256 rows
    int capacity;        // planes that have memory
    int width;           // 16, 32, 64 or 128
};
constexpr int MAX_ADAPTERS = 1024, SORT_THREADS = 1024;

// Exclusive prefix sum over one value per thread of a 1024-thread block; `all` their sum.
__device__ __forceinline__ int block_prefix(int v, int *warp_sum, int &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int sum = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    const int w = warp_sum[lane];
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
    all = __reduce_add_sync(0xffffffffu, w);
    return before + sum - v;
}

// The group of place `t` given the groups' first places (n + 1 of them, ascending).
__device__ __forceinline__ int group_at(const int *first, int n, int t) {
    int lo = 0, hi = n;   // first[lo] <= t < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        (first[mid] <= t ? lo : hi) = mid;
    }
    return lo;
}

// Groups (or -1: none) of rows 256 t + 32 i + lane; -2 past the end.
__device__ __forceinline__ void load_groups(int M, const Adapters &ad, const unsigned char *no_rank, int t, int (&b)[8]) {
    const long long r0 = (long long)t * 256 + (threadIdx.x & 31);
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = r0 + 32 * i < M ? ad.of_row(r0 + 32 * i) : -2;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (b[i] >= 0 && no_rank[b[i]]) b[i] = -1;
}

// For each 256 rows the adapters that they use, in ascending order, their planes, and
// which of them each row uses.  A warp to 256 rows, by a bit for each adapter.
__device__ __forceinline__ void lay_out_planes(int M, const Adapters &ad, const Groups &g, const unsigned char *no_rank,
                                               int *sm, int *warp_sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, a = threadIdx.x, tiles = (M + 255) / 256;
    int *bits = sm + warp * 32, *used = sm + 32 * 32;
    used[a] = 0;
    __syncthreads();
    const int per_plane = g.width >= 64 ? 1 : 64 / g.width, halves = g.width > 64 ? g.width / 64 : 1;
    for (int t = warp; t < tiles; t += 32) {
        int b[8];
        load_groups(M, ad, no_rank, t, b);
        bits[lane] = 0;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const unsigned same = __match_any_sync(0xffffffffu, b[i]);
            if (b[i] >= 0 && (same & ((1u << lane) - 1)) == 0) {
                atomicOr(&bits[b[i] >> 5], 1 << (b[i] & 31));
                used[b[i]] = 1;
            }
        }
        __syncwarp();
        // word w of the bits is lane w's; below: adapters in the words before it
        const unsigned word = unsigned(bits[lane]);
        int below = __popc(word);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, below, o);
            if (lane >= o) below += u;
        }
        const int kinds = __shfl_sync(0xffffffffu, below, 31), planes = (kinds * g.width + 63) / 64;
        below -= __popc(word);
        if (lane == 0) g.planes[t] = make_int4(0, planes, 0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int w = max(b[i], 0) >> 5 & 31;
            const unsigned of_w = __shfl_sync(0xffffffffu, word, w);
            const int position = __shfl_sync(0xffffffffu, below, w) + __popc(of_w & ((1u << (b[i] & 31)) - 1));
            if (b[i] > -2 && SG_IN_RANGE((long long)t * 256 + i * 32 + lane < M && position >= 0 && position <= kinds))
                g.position[t * 256 + i * 32 + lane] = b[i] >= 0 ? position : 0;
        }
        int4 *list = g.plane_adapter + (long long)t * g.most_planes;
        unsigned left = word;
        for (int k = below; left != 0; ++k, left &= left - 1) {
            const int id = lane * 32 + __ffs(left) - 1;
            if (!SG_IN_RANGE(k * g.width / 64 < planes && (k + 1) * g.width <= g.most_planes * 64 && id < ad.L)) break;
            if (g.width >= 64) {
                for (int h = 0; h < halves; ++h) list[k * halves + h] = make_int4(id, h * 64, 0, 0);
            } else {
                int *to = reinterpret_cast<int *>(&list[k / per_plane]);
                to[k % per_plane] = id;
                if (k == kinds - 1)
                    for (int d = k % per_plane + 1; d < per_plane; ++d) to[d] = id;
            }
        }
        __syncwarp();
    }
    __syncthreads();
    if (a < ad.L) g.used[a] = used[a], g.unclean[a] = 0;
    int all;
    for (int base = 0, t = 0; t < tiles; t += SORT_THREADS, base += all) {   // first planes of the tiles
        const int n = t + a < tiles ? g.planes[t + a].y : 0;
        const int p = base + block_prefix(n, warp_sum, all);
        if (t + a < tiles) g.planes[t + a] = make_int4(p, n, p + n <= g.capacity, 0);
    }
}

// The counting sort: each warp walks its share of the rows twice, 256 at a time.
__device__ __forceinline__ void sort_rows(int M, const Adapters &ad, const Groups &g, const unsigned char *no_rank, int *sm,
                                          int *warp_sum) {
    const int L = ad.L, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, a = threadIdx.x;
    int *count = sm;                       // [warp][group], then the next place of each
    int *first = count + 32 * (L + 1);     // L + 2: first place of a group
    int *chunk0 = first + (L + 2);
    for (int i = threadIdx.x; i < 32 * (L + 1); i += SORT_THREADS) count[i] = 0;
    __syncthreads();
    const int tiles = (M + 255) / 256, per = (tiles + 31) / 32;
    const int t0 = min(warp * per, tiles), t1 = min(t0 + per, tiles);
    int *mine = count + warp * (L + 1);
    for (int t = t0; t < t1; ++t) {
        int b[8];
        load_groups(M, ad, no_rank, t, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int group = b[i] == -1 ? L : b[i];
            const unsigned same = __match_any_sync(0xffffffffu, group);
            if (group >= 0 && (same & ((1u << lane) - 1)) == 0) mine[group] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    // first places of the groups (up to 1025 of them: group L by the last thread alone)
    int rows = 0, all;
    if (a < L)
        for (int w = 0; w < 32; ++w) rows += count[w * (L + 1) + a];
    const int at = block_prefix(rows, warp_sum, all);
    if (a < L) first[a] = at;
    if (a == SORT_THREADS - 1) first[L] = at + rows, first[L + 1] = M;
    const int chunk_at = block_prefix((rows + g.chunk - 1) / g.chunk, warp_sum, all);
    if (a < L) chunk0[a] = chunk_at;
    if (a == SORT_THREADS - 1) chunk0[L] = all;
    __syncthreads();
    for (int b = threadIdx.x; b <= L; b += SORT_THREADS) {
        g.chunk_begin[b] = chunk0[b];
        int place = first[b];
        for (int w = 0; w < 32; ++w) {
            const int n = count[w * (L + 1) + b];
            count[w * (L + 1) + b] = place;
            place += n;
        }
    }
    __syncthreads();
    for (int t = t0; t < t1; ++t) {
        int b[8];
        load_groups(M, ad, no_rank, t, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int group = b[i] == -1 ? L : b[i];
            const unsigned same = __match_any_sync(0xffffffffu, group);
            const int before = __popc(same & ((1u << lane) - 1));
            const int place = group >= 0 ? mine[group] + before : 0;
            __syncwarp();
            if (group >= 0) {
                if (SG_IN_RANGE(place >= 0 && place < M)) g.perm[place] = t * 256 + i * 32 + lane;
                if (before == 0) mine[group] += __popc(same);
            }
            __syncwarp();
        }
    }
    for (int t = threadIdx.x; t < g.max_chunks; t += SORT_THREADS) {
        if (t >= chunk0[L]) {
            g.chunks[t] = make_int4(-1, 0, 0, 0);
            continue;
        }
        const int b = group_at(chunk0, L, t), p = first[b] + (t - chunk0[b]) * g.chunk;
        const int n = min(g.chunk, first[b + 1] - p);
        const bool in = SG_IN_RANGE(chunk0[L] <= g.max_chunks && p >= 0 && n > 0 && (long long)p + n <= M);
        g.chunks[t] = make_int4(b, p, in ? n : 0, 0);
    }
}

constexpr size_t sort_smem(int L) {
    const size_t sort = size_t(32) * (L + 1) + 2 * (L + 2), planes = 32 * 32 + SORT_THREADS;
    return (sort > planes ? sort : planes) * 4;
}

// Block 0 lays the planes out; block 1, where there is one, sorts the rows.  Bound by
// latency: 6 us up to 8192 rows.
__global__ void __launch_bounds__(SORT_THREADS, 1) group_rows_kernel(int M, Adapters ad, Groups g) {
    extern __shared__ int sm[];
    __shared__ int warp_sum[32];
    __shared__ unsigned char no_rank[MAX_ADAPTERS];
    sg::wait_prerequisites();
    sg::launch_dependents();
    if (int(threadIdx.x) < ad.L) no_rank[threadIdx.x] = ad.rank(threadIdx.x) == 0;
    __syncthreads();
    if (blockIdx.x == 0)
        lay_out_planes(M, ad, g, no_rank, sm, warp_sum);
    else
        sort_rows(M, ad, g, no_rank, sm, warp_sum);
}

// One side of the stack laid out for the tensor cores: the parts of the used adapters as
// planes part * L + a of width x cols, zero past the adapter's rank.  `trans`: V_a is
// stored cols x R, else R x cols.  `watch`: it enters the rank-side planes, where what is
// not finite would reach other adapters' rows: unclean[a] says that there is some.
template <class T>
struct StackSide {
    Stack<const T> V;
    int cols;
    bool trans, watch;
    Parts to;
};

// A block to 8 rank columns (blockIdx.z) x 256 columns of an adapter of either side (`across`
// blocks of the first, the rest of the second): a warp to 8 x 32, a thread to eight columns
// of one, so that loads and stores cover 16 bytes and 64 without shared memory.
template <class T>
__global__ void __launch_bounds__(256)
    pack_stack_kernel(StackSide<T> first, StackSide<T> second, int across, Adapters ad, Groups g) {
    constexpr int PARTS = sizeof(T) == 4 ? 3 : 1;
    sg::wait_prerequisites();
    sg::launch_dependents();
    const int a = blockIdx.y;
    const bool is_first = int(blockIdx.x) < across;
    const StackSide<T> &side = is_first ? first : second;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cols = side.cols;
    const int c = (int(blockIdx.x) - (is_first ? 0 : across)) * 256 + warp * 32 + (lane >> 3) * 8;
    const int rank = ad.rank(a);
    if (!g.used[a] || c >= cols) return;
    const T *v = side.V.matrix(a);
    const long long ld = side.V.ld, step = side.trans ? ld : 1;   // from column to column
    Parts at = side.to;
    at.p += a * at.plane;
    at.plane *= ad.L;
    const int r = blockIdx.z * 8 + (lane & 7);
    if (!SG_IN_RANGE(a < ad.L && c >= 0 && c + 8 <= at.pitch && (r + 1) * at.pitch <= side.to.plane)) return;
    const T *p = v + (side.trans ? c * ld + r : r * ld + c);
    bool finite = true;
    float x[8];
#pragma unroll
    for (int d = 0; d < 8; ++d) {
        x[d] = c + d < cols && r < rank ? to_f32(p[d * step]) : 0.0f;
        finite = finite && isfinite(x[d]);
    }
    store_parts<PARTS>(at, r, c, x);
    if (side.watch && !finite) g.unclean[a] = 1;
}

}  // namespace sgl
