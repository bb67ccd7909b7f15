// norm.cuh -- kernels of the root-mean-square norm and of rows in 8 bits.
//
//   v = x + r, held in the call's type;   y_j = v_j rstd w_j,  rstd = 1 / sqrt(mean(v^2) + eps)
//   8 bits: scale = max|y| / 127,  q_j = rint(y_j / scale) = rint(127 p_j / max|p|),  p = v w
//
// q does not depend on rstd, so the row's sum of squares and its largest |p| are taken together in
// one pass, and q is the exactly rounded quotient whatever order the sum is taken in (rows8.cuh; p has
// 16 bits from bfloat16, 48 from float32, where the maximum is kept as a pair, value and remainder,
// for the comparison near a tie).
//
// A row goes to a group of threads (a warp or a block) that keeps it in registers between its
// two uses, up to 16384 columns; longer rows are read twice (LONG).  Everything is read and
// written once, and the kernels are bound by that.
#pragma once

#include "kernels.cuh"
#include "rows8.cuh"

namespace sgl {

// The range of a row's sum of squares in which no term has overflowed or counts for too little.
constexpr float LEAST_SQUARES = 0x1p-80f, MOST_SQUARES = 0x1p120f;

__host__ __device__ constexpr int norm_block(int threads) { return threads < 128 ? 256 : threads; }

// Where eight elements `c` of thread `t` lie in a row: 16 bytes together, next to the other threads'
// (WIDE, rows that are 16-byte aligned and of a multiple of 8 columns; float32: in two such pieces), or
// one by one, a group's width apart.
template <class T, int THREADS, bool WIDE>
struct Place {
    static constexpr int PER = WIDE ? 16 / int(sizeof(T)) : 1;   // together
    int K, base, t;

    __device__ int column(int c, int e) const { return base + ((c * (8 / PER) + e / PER) * THREADS + t) * PER + e % PER; }
    __device__ void load(const T *row, int c, float (&v)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; e += PER) {
            const int j = column(c, e);
            if constexpr (PER == 8) {
                if (j < K) load8(row + j, v);
            } else if constexpr (PER == 4) {
                float x[4];
                if (j < K) load4(row + j, x);
#pragma unroll
                for (int d = 0; d < 4; ++d) v[e + d] = j < K ? x[d] : 0.0f;
            } else {
                v[e] = j < K ? to_f32(row[j]) : 0.0f;
            }
            if (PER == 8 && j >= K)
#pragma unroll
                for (int d = 0; d < 8; ++d) v[d] = 0.0f;
        }
    }
    __device__ void store(T *row, int c, const float (&v)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; e += PER) {
            const int j = column(c, e);
            if (j >= K) continue;
            if constexpr (PER == 8) {
                store8(row + j, v);
            } else if constexpr (PER == 4) {
                const float x[4] = {v[e], v[e + 1], v[e + 2], v[e + 3]};
                store4(row + j, x);
            } else {
                row[j] = from_f32<T>(v[e]);
            }
        }
    }
    // Eight integers of at most 127 in magnitude, given as floats.
    __device__ void store_q(signed char *row, int c, const float (&r)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; e += PER) {
            const int j = column(c, e);
            if (j >= K) continue;
            if constexpr (PER == 8)
                *reinterpret_cast<uint2 *>(row + j) = make_uint2(pack_s8(r, 1.0f), pack_s8(r + 4, 1.0f));
            else if constexpr (PER == 4)
                *reinterpret_cast<uint32_t *>(row + j) = pack_s8(r + e, 1.0f);
            else
                row[j] = static_cast<signed char>(__float2int_rn(r[e]));
        }
    }
};

// ------------------------------------------------------------------ a group's sums and maxima
// A product's magnitude exactly: `hi` its fp32 value, `lo` what that leaves (bfloat16: nothing).
struct Top {
    uint32_t hi;   // bits of a magnitude: they order as it does, an infinity or a NaN above all
    float lo;

    __device__ bool below(const Top &o) const { return hi < o.hi || (hi == o.hi && lo < o.lo); }
    __device__ float value() const { return __uint_as_float(hi); }
};
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <bool WITH_LO>
__device__ __forceinline__ Top warp_top(Top t) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, t.hi);
    if (WITH_LO) t.lo = from_ordered(__reduce_max_sync(0xffffffffu, t.hi == hi ? ordered(t.lo) : 0u));
    t.hi = hi;
    return t;
}

// Added up in pairs, so that few roundings follow one another in a row's sum (1 x 8192: 5.5e-8 from 64 bits, in a
// chain 6.6e-8).
__device__ __forceinline__ float sum_of_squares(const float (&v)[8]) {
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = fmaf(v[i + 4], v[i + 4], v[i] * v[i]);
    return (s[0] + s[2]) + (s[1] + s[3]);
}

// Two sums and a maximum over a group, the warps' in a fixed order.  `turn` alternates from call to
// call: a warp writes here again only when all have read what it wrote the time before.
struct GroupSums {
    float a[2][32], b[2][32], lo[2][32];
    uint32_t hi[2][32];
    double wide[32];
};
template <int THREADS, bool B, bool TOP, bool WITH_LO>
__device__ __forceinline__ void group_reduce(GroupSums &sm, int turn, float &a, float &b, Top &top) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    a = warp_sum(a);
    if (B) b = warp_sum(b);
    if (TOP) top = warp_top<WITH_LO>(top);
    if (THREADS == 32) return;
    if (lane == 0) {
        sm.a[turn][warp] = a;
        if (B) sm.b[turn][warp] = b;
        if (TOP) sm.hi[turn][warp] = top.hi, sm.lo[turn][warp] = top.lo;
    }
    __syncthreads();
    // 16 and 32 warps' by a tree in every warp (1 x 4096 in 8 bits with residual 4.5 -> 3.0 us), fewer one after the other (y
    // from 8192 x 2048 bfloat16 15.3, by the tree 15.8; in 8 bits it would be 24.4 for 25.9, but y is the same bits with
    // and without them; the backward pass at any width)
    if constexpr (THREADS >= 512 && !B) {
        const bool in = lane < THREADS / 32;
        a = warp_sum(in ? sm.a[turn][lane] : 0.0f);
        if (TOP) top = warp_top<WITH_LO>(in ? Top{sm.hi[turn][lane], sm.lo[turn][lane]} : Top{0, 0.0f});
        return;
    }
    a = b = 0.0f;
    top = Top{0, 0.0f};
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        a += sm.a[turn][w];
        if (B) b += sm.b[turn][w];
        if (TOP) {
            const Top o{sm.hi[turn][w], sm.lo[turn][w]};
            if (top.below(o)) top = o;
        }
    }
}
template <int THREADS>
__device__ __forceinline__ void group_sync() {
    if (THREADS == 32) __syncwarp();
    else __syncthreads();
}
template <int THREADS>
__device__ __forceinline__ double group_sum(GroupSums &sm, double v) {
    v = warp_sum(v);
    if (THREADS == 32) return v;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm.wide[threadIdx.x >> 5] = v;
    __syncthreads();
    double all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) all += sm.wide[w];
    return all;
}
template <int THREADS>
__device__ __forceinline__ double group_max(GroupSums &sm, double v) {   // of magnitudes, NaN the largest
    auto larger = [](double a, double b) { return a != a || a > b ? a : b; };
#pragma unroll
    for (int o = 16; o; o >>= 1) v = larger(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (THREADS == 32) return v;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm.wide[threadIdx.x >> 5] = v;
    __syncthreads();
    double all = sm.wide[0];
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w) all = larger(all, sm.wide[w]);
    return all;
}

enum NormKind { NORM, NORM8, ROWS8 };   // y alone; q and, where Y is given, y; q of x itself

// ------------------------------------------------------------------ rows out of fp32's range
// tie_exact (rows8.cuh) of a product p of float32 values, of 48 bits as `top` is, in 64: (n + 1/2) top has 56, so the
// comparison takes what its rounding leaves into account.  Near a tie 127 |p| - t is under 2^-13 top and a whole number
// of the smaller of the two products' last places, which then is under 2^44 of them: both differences are exact.
__device__ __forceinline__ double tie_of(double p, double quotient, double top) {
    const double n = floor(fabs(quotient)), h = n + 0.5, t = h * top;
    const double d = fma(127.0, fabs(p), -t) - fma(h, top, -t);
    const bool odd = (int(n) & 1) != 0;
    return copysign(d > 0 || (d == 0 && odd) ? n + 1.0 : n, quotient);
}
static __device__ __noinline__ float tie_wide(float v, float w, float quotient, float top_hi, float top_lo) {
    return float(tie_of(double(v) * w, quotient, double(top_hi) + top_lo));
}

// A row's q and the largest |p| in 64 bits, where products leave fp32's range.
template <class T, int THREADS, bool WEIGHED, class V>
__device__ __forceinline__ double rare_rows8(GroupSums &sm, V v, const T *w, signed char *q, int K, int t) {
    double top = 0;
    bool any = false;   // rows of zeros, padding, need no more than this pass
    for (int j = t; j < K; j += THREADS) {
        const float x = v(j), y = WEIGHED ? to_f32(w[j]) : 1.0f;
        if (x == 0.0f && y - y == 0.0f) continue;
        any = true;
        const double p = fabs(double(x) * y);
        top = p != p || p > top ? p : top;
    }
    any = THREADS == 32 ? __any_sync(0xffffffffu, any) : __syncthreads_or(any);
    if (any) top = group_max<THREADS>(sm, top);
    if (!any || !(top > 0 && top <= 1.7e308)) {   // zeros, an infinity or a NaN
        for (int j = t; j < K; j += THREADS) q[j] = 0;
        return top;
    }
    for (int j = t; j < K; j += THREADS) {
        const double p = double(v(j)) * (WEIGHED ? to_f32(w[j]) : 1.0f), quotient = 127.0 * p / top;
        const float near = whole(float(quotient));
        q[j] = static_cast<signed char>(fabsf(float(quotient) - near) > 0.5f - NEAR ? tie_of(p, quotient, top) : near);
    }
    return top;
}

// 1 / sqrt(mean(v^2) + eps) where the squares leave fp32's range, and rstd with them: it is up to 2^165 where v is
// subnormal and eps is 0.  As r * s, s a power of two, r a normal number: v s r is rounded once, as v rstd is in other
// rows.  An infinity in v makes it 0, a NaN a NaN.
struct RareRstd {
    float r, s;
};
template <int THREADS, class V>
__device__ __forceinline__ RareRstd rare_rstd(GroupSums &sm, V v, int K, float eps, int t) {
    double ss = 0;
    for (int j = t; j < K; j += THREADS) ss += double(v(j)) * v(j);
    const double rstd = 1.0 / sqrt(group_sum<THREADS>(sm, ss) / K + eps);
    const float s = rstd > 0x1p64 ? 0x1p64f : rstd < 0x1p-64 ? 0x1p-64f : 1.0f;
    return {float(rstd / s), s};
}

// A row whose squares (`far`) or products leave fp32's range, all that is left of it.  (Nothing of the row is needed after
// this call, so that the registers that it takes cost other rows none.)
template <class T, int KIND, int THREADS, class V>
__device__ __noinline__ void rare_row(GroupSums &sm, V v, const T *w, T *y, signed char *q, float *scale, int K, float eps, int t,
                                      bool far, float rstd) {
    RareRstd at{rstd, 1.0f};
    if (KIND != ROWS8 && far) at = rare_rstd<THREADS>(sm, v, K, eps, t);
    if (KIND != NORM) {
        const double top = rare_rows8<T, THREADS, KIND != ROWS8>(sm, v, w, q, K, t);
        if (t == 0) *scale = top <= 1.7e308 ? float(top * at.s * at.r / 127.0) : __uint_as_float(0x7fc00000u);
    }
    if (KIND != ROWS8 && y)   // (y may be X: an element's own reads are done)
        for (int j = t; j < K; j += THREADS) y[j] = from_f32<T>(v(j) * at.s * at.r * to_f32(w[j]));
}

// ------------------------------------------------------------------ forward
template <class T>
struct NormCall {
    int M, K;
    const T *X, *R, *w;
    T *S, *Y;
    signed char *q;
    float *scale;
    long long ldx, ldr, lds, ldy, ldq;
    float eps;
};

template <class T, int KIND, int THREADS, int CHUNKS, bool WIDE, bool LONG>
__global__ void __launch_bounds__(norm_block(THREADS))
    norm_kernel(const NormCall<T> a) {
    constexpr int GROUPS = norm_block(THREADS) / THREADS, SPAN = THREADS * 8 * CHUNKS;
    constexpr bool EIGHT = KIND != NORM, WITH_LO = EIGHT && KIND != ROWS8 && sizeof(T) == 4;
    __shared__ GroupSums sm;
    sg::wait_prerequisites();
    sg::launch_dependents();
    const int t = threadIdx.x % THREADS;
    const long long row = (long long)blockIdx.x * GROUPS + threadIdx.x / THREADS;
    if (row >= a.M || !SG_IN_RANGE(LONG || a.K <= SPAN)) return;
    const T *x = a.X + row * a.ldx, *r = a.R ? a.R + row * a.ldr : nullptr;
    T *s = a.S ? a.S + row * a.lds : nullptr, *y = KIND != ROWS8 && a.Y ? a.Y + row * a.ldy : nullptr;
    signed char *q = EIGHT ? a.q + row * a.ldq : nullptr;

    float v[CHUNKS][8], w[8];
    auto read = [&](const Place<T, THREADS, WIDE> &at, bool again) {
        const T *from = again && s ? s : x;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) at.load(from, c, v[c]);
        if constexpr (KIND != ROWS8) {
            if (!r || (again && s)) return;
            float u[CHUNKS][8];
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) at.load(r, c, u[c]);
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[c][e] = to_f32(from_f32<T>(v[c][e] + u[c][e]));
        }
    };

    float squares = 0.0f, none = 0.0f;
    Top top{0, 0.0f};
    for (int base = 0; base < (LONG ? a.K : 1); base += SPAN) {
        const Place<T, THREADS, WIDE> at{a.K, base, t};
        read(at, false);
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            if (KIND != ROWS8 && s) at.store(s, c, v[c]);
            if (EIGHT && KIND != ROWS8) at.load(a.w, c, w);
            if (KIND != ROWS8) squares += sum_of_squares(v[c]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (EIGHT) {
                    const float p = KIND == ROWS8 ? v[c][e] : v[c][e] * w[e];
                    Top o{magnitude_bits(p), 0.0f};
                    if (WITH_LO) {
                        o.lo = fmaf(v[c][e], w[e], -p);
                        o.lo = p < 0.0f ? -o.lo : o.lo;
                        if (top.below(o)) top = o;
                    } else {
                        top.hi = max(top.hi, o.hi);
                    }
                }
            }
        }
    }
    group_reduce<THREADS, false, EIGHT, WITH_LO>(sm, 0, squares, none, top);

    if (THREADS == 32) __syncwarp();   // (else group_reduce's barrier)
    auto held = [&](int j) {   // v, from what any thread may have written of it above
        if (KIND == ROWS8) return to_f32(x[j]);
        return s ? to_f32(s[j]) : r ? to_f32(from_f32<T>(to_f32(x[j]) + to_f32(r[j]))) : to_f32(x[j]);
    };
    float rstd = 1.0f, times = 0.0f;   // times: 127 / max|p|
    bool far = false;
    if (KIND != ROWS8) {
        rstd = 1.0f / sqrtf(squares / float(a.K) + a.eps);
        far = !(squares <= MOST_SQUARES) || (squares < LEAST_SQUARES && a.eps < 1e-10f);
    }
    if (far || (EIGHT && !(top.value() >= LEAST_TOP && top.value() <= MOST_TOP))) {
        rare_row<T, KIND, THREADS>(sm, held, a.w, y, q, EIGHT ? a.scale + row : nullptr, a.K, a.eps, t, far, rstd);
        return;
    }
    if (EIGHT) {
        times = 127.0f / top.value();
        if (t == 0) a.scale[row] = (KIND == ROWS8 ? top.value() : top.value() * rstd) / 127.0f;
    }

    for (int base = 0; base < (LONG ? a.K : 1); base += SPAN) {
        const Place<T, THREADS, WIDE> at{a.K, base, t};
        if (LONG) read(at, true);
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            float out[8];
            if (KIND != ROWS8) at.load(a.w, c, w);
            if (EIGHT) {
                float off = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float quotient = (KIND == ROWS8 ? v[c][e] : v[c][e] * w[e]) * times;
                    out[e] = whole(quotient);
                    off = fmaxf(off, fabsf(quotient - out[e]));
                }
                if (off > 0.5f - NEAR) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float p = KIND == ROWS8 ? v[c][e] : v[c][e] * w[e], quotient = p * times;
                        if (fabsf(quotient - out[e]) > 0.5f - NEAR)
                            out[e] = WITH_LO ? tie_wide(v[c][e], w[e], quotient, top.value(), top.lo)
                                             : tie_exact(p, quotient, top.value());
                    }
                }
                at.store_q(q, c, out);
            }
            if (KIND != ROWS8 && y) {
#pragma unroll
                for (int e = 0; e < 8; ++e) out[e] = v[c][e] * rstd * w[e];
                at.store(y, c, out);
            }
        }
    }
}

// ------------------------------------------------------------------ backward
// With n = v rstd, g = dy w and c = sum(g n) / K:  dx = ds + rstd (g - c n),  dw = sum over rows of dy n.
// A group keeps the sums of dw's columns over its rows, which are `groups` apart; a second
// kernel adds the groups' (of a block's warps: the block's) in order.
template <class T>
struct NormBackCall {
    int M, K;
    const T *dY, *V, *w, *dS;
    T *dX;
    float *partial;   // blocks x K, or null: no dw
    long long lddy, ldv, ldds, lddx;
    float eps;
};

// The same of the backward pass, where the row's work goes on.
template <class T, int THREADS>
__device__ __noinline__ RareRstd rare_row_rstd(GroupSums &sm, const T *v, int K, float eps, int t) {
    return rare_rstd<THREADS>(sm, [&](int j) { return to_f32(v[j]); }, K, eps, t);
}

// The rows to come stand in a ring of asynchronous copies, each thread's own elements in its own
// slots, so that they need no barrier; bfloat16 rows that are not 16-byte aligned, and rows that
// are too long for a ring of two, go from memory to registers.
template <class T, int THREADS, int CHUNKS, bool WIDE, bool LONG>
struct NormRing {
    static constexpr size_t STAGE = size_t(3) * CHUNKS * 8 * sizeof(T) * norm_block(THREADS), MOST = 98304;
    static constexpr bool ON = !LONG && (WIDE || sizeof(T) == 4) && STAGE <= MOST;
    static constexpr int DEPTH = !ON ? 1 : STAGE * 4 <= MOST ? 4 : STAGE * 3 <= MOST ? 3 : 2;
    static constexpr size_t BYTES = ON ? DEPTH * STAGE : 0;
};
template <int THREADS, int CHUNKS>
constexpr int norm_blocks_per_sm = THREADS == 128 ? 6 : THREADS == 512 ? 1 : 2;

template <class T, int THREADS, int CHUNKS, bool WIDE, bool LONG>
__global__ void __launch_bounds__(norm_block(THREADS), norm_blocks_per_sm<THREADS, CHUNKS>)
    norm_backward_kernel(const NormBackCall<T> a) {
    constexpr int BLOCK = norm_block(THREADS), GROUPS = BLOCK / THREADS, SPAN = THREADS * 8 * CHUNKS;
    using Ring = NormRing<T, THREADS, CHUNKS, WIDE, LONG>;
    constexpr bool KEEP_W = !LONG && CHUNKS <= 2;
    extern __shared__ __align__(16) unsigned char norm_ring[];
    __shared__ GroupSums sm;
    sg::wait_prerequisites();
    sg::launch_dependents();
    __shared__ float columns[GROUPS > 1 ? SPAN : 1];
    const int t = threadIdx.x % THREADS, group = threadIdx.x / THREADS;
    if (!SG_IN_RANGE(LONG || a.K <= SPAN)) return;
    float *partial = a.partial ? a.partial + (long long)blockIdx.x * a.K : nullptr;
    const long long step = (long long)gridDim.x * GROUPS;
    long long row = (long long)blockIdx.x * GROUPS + group;

    // Element e of chunk c of matrix m: 16 bytes at a time, or one by one next to the other threads'.
    auto slot = [&](int stage, int m, int c, int e) {
        constexpr int PER = 16 / int(sizeof(T));
        const int at = ((stage * 3 + m) * CHUNKS + c) * 8;
        return reinterpret_cast<T *>(norm_ring) +
               (WIDE ? (at + e / PER * PER) * BLOCK + int(threadIdx.x) * PER + e % PER : (at + e) * BLOCK + int(threadIdx.x));
    };
    auto issue = [&](int stage, long long r) {
        if constexpr (Ring::ON) {
            const Place<T, THREADS, WIDE> at{a.K, 0, t};
            if (r < a.M)
#pragma unroll
                for (int m = 0; m < 3; ++m) {
                    const T *p = m == 0 ? a.V + r * a.ldv : m == 1 ? a.dY + r * a.lddy : a.dS + r * a.ldds;
                    if (m == 2 && !a.dS) break;
#pragma unroll
                    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
                        for (int e = 0; e < 8; e += WIDE ? 16 / int(sizeof(T)) : 1) {
                            const uint32_t to = sg::smem_addr(slot(stage, m, c, e));
                            const bool in = at.column(c, e) < a.K;
                            const T *from = in ? p + at.column(c, e) : p;
                            if constexpr (WIDE) sg::cp_async16(to, from, in ? 16u : 0u);
                            else sg::cp_async4(to, from, in ? 4u : 0u);
                        }
                }
            sg::cp_async_commit();
        }
    };
    auto take = [&](int stage, int m, int c, float (&x)[8]) {
        if constexpr (WIDE && sizeof(T) == 4) {
            float lo[4], hi[4];
            load4(slot(stage, m, c, 0), lo);
            load4(slot(stage, m, c, 4), hi);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = lo[e], x[e + 4] = hi[e];
        } else if constexpr (WIDE) {
            load8(slot(stage, m, c, 0), x);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = to_f32(*slot(stage, m, c, e));
        }
    };

    float v[CHUNKS][8], dy[CHUNKS][8], dw[LONG ? 1 : CHUNKS][8] = {}, w[KEEP_W ? CHUNKS : 1][8];
    auto weight = [&](const Place<T, THREADS, WIDE> &at, int c) -> float(&)[8] {
        if (!KEEP_W) at.load(a.w, c, w[0]);
        return w[KEEP_W ? c : 0];
    };
#pragma unroll
    for (int c = 0; KEEP_W && c < CHUNKS; ++c) Place<T, THREADS, WIDE>{a.K, 0, t}.load(a.w, c, w[c]);
#pragma unroll
    for (int d = 0; Ring::ON && d < Ring::DEPTH; ++d) issue(d, row + d * step);
    int turn = 0, stage = 0;
    bool first = true;
    for (; row < a.M; row += step) {
        const T *vr = a.V + row * a.ldv, *dyr = a.dY + row * a.lddy, *dsr = a.dS ? a.dS + row * a.ldds : nullptr;
        T *dxr = a.dX + row * a.lddx;
        auto read = [&](const Place<T, THREADS, WIDE> &at) {
            if constexpr (Ring::ON) sg::cp_async_wait<Ring::DEPTH - 1>();
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
                if constexpr (Ring::ON)
                    take(stage, 0, c, v[c]), take(stage, 1, c, dy[c]);
                else
                    at.load(vr, c, v[c]), at.load(dyr, c, dy[c]);
            }
        };
        auto scale_v = [&](float by) {
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[c][e] *= by;
        };
        float squares = 0.0f, gv = 0.0f;
        Top none{};
        for (int base = 0; base < (LONG ? a.K : 1); base += SPAN) {
            const Place<T, THREADS, WIDE> at{a.K, base, t};
            read(at);
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
                const float(&u)[8] = weight(at, c);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    squares = fmaf(v[c][e], v[c][e], squares);
                    gv = fmaf(dy[c][e] * u[e], v[c][e], gv);
                }
            }
        }
        group_reduce<THREADS, true, false, false>(sm, turn, squares, gv, none);
        turn ^= 1;
        float rstd = 1.0f / sqrtf(squares / float(a.K) + a.eps), mean = gv * rstd / float(a.K), shift = 1.0f;
        // (the products' sum may leave the range where the squares do not; a NaN comes through in either way)
        if (!(squares <= MOST_SQUARES) || (squares < LEAST_SQUARES && a.eps < 1e-10f) || !(fabsf(mean) <= 0x1.fffffep127f)) {
            double sum = 0;
            for (int j = t; j < a.K; j += THREADS) sum += double(to_f32(dyr[j])) * to_f32(a.w[j]) * to_f32(vr[j]);
            const RareRstd of = rare_row_rstd<T, THREADS>(sm, vr, a.K, a.eps, t);
            rstd = of.r, shift = of.s;
            mean = float(group_sum<THREADS>(sm, sum) * shift * rstd / a.K);
            group_sync<THREADS>();   // dX, written below, may be dY
            if (!LONG) scale_v(shift);
        }
        for (int base = 0; base < (LONG ? a.K : 1); base += SPAN) {
            const Place<T, THREADS, WIDE> at{a.K, base, t};
            if (LONG) {
                read(at);
                if (shift != 1.0f) scale_v(shift);
            }
            float ds[CHUNKS][8];
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
                if (!dsr) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) ds[c][e] = 0.0f;
                } else if constexpr (Ring::ON) {
                    take(stage, 2, c, ds[c]);
                } else {
                    at.load(dsr, c, ds[c]);
                }
            }
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
                const float(&u)[8] = weight(at, c);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float n = v[c][e] * rstd;   // (shift: 1 but for rows out of range, whose v holds it too)
                    ds[c][e] = fmaf(rstd, fmaf(-mean, n, dy[c][e] * u[e]) * shift, ds[c][e]);
                    if (!LONG) {
                        dw[c][e] = fmaf(dy[c][e], n, dw[c][e]);
                    } else if (partial && at.column(c, e) < a.K) {   // (this thread's own column)
                        float *p = partial + at.column(c, e);
                        *p = fmaf(dy[c][e], n, first ? 0.0f : *p);
                    }
                }
                at.store(dxr, c, ds[c]);
            }
        }
        issue(stage, row + Ring::DEPTH * step);
        stage = stage + 1 == Ring::DEPTH ? 0 : stage + 1;
        first = false;
    }
    if constexpr (Ring::ON) sg::cp_async_wait<0>();
    if (LONG || !partial) return;
    const Place<T, THREADS, WIDE> at{a.K, 0, t};
    for (int g = 0; g < GROUPS; ++g) {   // a block's warps in order
        if (GROUPS > 1) __syncthreads();
        if (group != g) continue;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int j = at.column(c, e);
                if (j >= a.K) continue;
                if (GROUPS == 1)
                    partial[j] = dw[c][e];
                else
                    columns[j] = g == 0 ? dw[c][e] : columns[j] + dw[c][e];
            }
    }
    if (GROUPS == 1) return;
    __syncthreads();
    for (int j = threadIdx.x; j < a.K; j += BLOCK) partial[j] = columns[j];
}

// dw from the blocks' sums: 32 columns to a block, its 32 warps' shares of the sums in order.
template <class T>
__global__ void __launch_bounds__(1024)
    norm_weight_kernel(int K, int sums, const float *__restrict__ partial, T *dw) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = blockIdx.x * 32 + lane;
    const int per = (sums + 31) / 32, last = min(sums, (warp + 1) * per);
    sg::wait_prerequisites();
    float s = 0.0f;
    if (j < K && SG_IN_RANGE(sums > 0)) {
#pragma unroll 8
        for (int i = warp * per; i < last; ++i) s += partial[(long long)i * K + j];
    }
    part[warp][lane] = s;
    __syncthreads();
    // a warp to a column: the shares by a tree
    const float all = warp_sum(part[lane][warp]);
    const int column = blockIdx.x * 32 + warp;
    if (lane == 0 && column < K) dw[column] = from_f32<T>(all);
}

}  // namespace sgl
