// act8.cu -- checkpoints of activations in 8 bits: the entry points that store
// them, read them back and take an activation's gradient from them.
//
// Each kernel makes one pass: every input and output byte moves once, and the
// arithmetic in between (a maximum over 32 columns, an exact scaling, for GELU
// one exponential and one reciprocal per element) runs in its shadow.
#include <algorithm>

#include "../../include/sgemm_layers.h"
#include "act8.cuh"
#include "activations.cuh"
#include "host_state.h"
#include "variant.cuh"

#define SGEMM_API extern "C" __attribute__((visibility("default")))

namespace {

using namespace sgl;

constexpr int kThreads = 256;

// ------------------------------------------------------------------ kernels
// What a kernel works on: `units` of 32 columns (wide forms) or 256, `per_row` to a row.
// (Rows by a division: GELU at 8192 x 16384 bfloat16 117 us, by multiplication 113.)
struct Blocks {
    unsigned units;
    Divisor per_row;
    int K;

#ifdef SGEMM_DEBUG_BOUNDS
    // Whether n columns from c of a row are the matrix's.
    __device__ bool holds(unsigned row, int c, int n) const {
        return row < units / per_row.d && c >= 0 && (long long)c + n <= K;
    }
#endif
};
struct Checkpoint {
    signed char *q, *e;
    long long ldq, lde;
};

// Wide form, for rows that are 16-byte aligned and of a multiple of 8 columns: a quarter
// of a block to a thread, its maximum over four lanes; so many blocks to a thread, all
// loaded before the first is used.  At 8192 x 16384, us (GB/s over the bytes of either
// side): bfloat16 store 68, with GELU 115 (5870), GELU gradient 111 (6080), load 67
// (6080); float32 with GELU 174 (6940), gradient 173.  What is left is issue slots: storing
// with half the depth 119, the gradient with two blocks to a thread 129, with four 151;
// reading back with one 72.
template <class T>
constexpr int kStoreDepth = sizeof(T) == 2 ? 4 : 2;
template <bool GRAD>
constexpr int kReadDepth = GRAD ? 1 : 2;

template <class T, int ACT, bool WITH_Y>
__global__ void __launch_bounds__(kThreads)
    store_wide_kernel(Blocks b, const T *Z, long long ldz, Checkpoint c, T *Y, long long ldy) {
    constexpr int D = kStoreDepth<T>;
    const int sub = threadIdx.x & 3;
    const unsigned first = (blockIdx.x * D) * (kThreads / 4) + (threadIdx.x >> 2);
    float z[D][8];
    unsigned row[D];
    int col[D];
    bool in[D];
#pragma unroll
    for (int d = 0; d < D; ++d) {
        const unsigned u = first + d * (kThreads / 4);
        row[d] = b.per_row.quotient(u);
        col[d] = int(u - row[d] * b.per_row.d) * ACT8_BLOCK + sub * 8;
        in[d] = u < b.units && col[d] < b.K && SG_IN_RANGE(b.holds(row[d], col[d], 8));
#pragma unroll
        for (int i = 0; i < 8; ++i) z[d][i] = 0.0f;
        if (in[d]) load8(Z + (long long)row[d] * ldz + col[d], z[d]);
    }
#pragma unroll
    for (int d = 0; d < D; ++d) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, magnitude_bits(z[d][i]));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = act8_exponent(top);
        if (!in[d]) continue;
        const float inverse = act8_inverse_step(e);
        uint32_t w[2] = {pack_s8(z[d], inverse), pack_s8(z[d] + 4, inverse)};
        if (e == ACT8_NAN || e == 121) {   // rare: nothing to keep, or 127 is exceeded
            w[0] = w[1] = 0;
            if (e == 121)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i / 4] |= (uint32_t(act8_quantise(z[d][i], inverse)) & 0xffu) << (8 * (i % 4));
        }
        *reinterpret_cast<uint2 *>(c.q + row[d] * c.ldq + col[d]) = make_uint2(w[0], w[1]);
        if (sub == 0) c.e[row[d] * c.lde + col[d] / ACT8_BLOCK] = static_cast<signed char>(e);
        if constexpr (WITH_Y) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 v = activate<T, ACT>(make_float2(z[d][i], z[d][i + 1]));
                y[i] = v.x, y[i + 1] = v.y;
            }
            store8(Y + (long long)row[d] * ldy + col[d], y);
        }
    }
}

// Any alignment and width: eight blocks of a row to a warp, a column of each to a lane, so
// that every access covers consecutive elements wherever the row starts.  GELU over 4097 x
// 3001 float32: 23 us stored, its gradient 23 (4900 GB/s; 25 with fewer than six thread blocks to an
// SM); one block to a warp took 41 and 39, most of it finding rows.
constexpr int kAnyDepth = 8;

template <class T, int ACT, bool WITH_Y>
__global__ void __launch_bounds__(kThreads)
    store_any_kernel(Blocks b, const T *Z, long long ldz, Checkpoint c, T *Y, long long ldy) {
    constexpr int D = kAnyDepth;
    const int lane = threadIdx.x & 31;
    const unsigned u = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), row = b.per_row.quotient(u);
    if (u >= b.units) return;
    const int c0 = int(u - row * b.per_row.d) * (D * ACT8_BLOCK) + lane;
    if (!SG_IN_RANGE(b.holds(row, c0 - lane, 1))) return;
    const T *zr = Z + (long long)row * ldz + c0;
    signed char *q = c.q + row * c.ldq + c0, *e = c.e + row * c.lde + (c0 - lane) / ACT8_BLOCK;
    T *y = WITH_Y ? Y + (long long)row * ldy + c0 : nullptr;
    float z[D];
#pragma unroll
    for (int d = 0; d < D; ++d) z[d] = c0 + d * ACT8_BLOCK < b.K ? to_f32(zr[d * ACT8_BLOCK]) : 0.0f;
    if constexpr (WITH_Y) {
#pragma unroll
        for (int d = 0; d < D; d += 2) {
            const float2 v = activate<T, ACT>(make_float2(z[d], z[d + 1]));
            if (c0 + d * ACT8_BLOCK < b.K) y[d * ACT8_BLOCK] = from_f32<T>(v.x);
            if (c0 + (d + 1) * ACT8_BLOCK < b.K) y[(d + 1) * ACT8_BLOCK] = from_f32<T>(v.y);
        }
    }
    // lane d works out the exponent of block d
    uint32_t top = 0;
#pragma unroll
    for (int d = 0; d < D; ++d) {
        const uint32_t t = __reduce_max_sync(0xffffffffu, magnitude_bits(z[d]));
        if (lane == d) top = t;
    }
    const int ex = act8_exponent(top);
    if (lane < D && c0 - lane + lane * ACT8_BLOCK < b.K) e[lane] = static_cast<signed char>(ex);
#pragma unroll
    for (int d = 0; d < D; ++d) {
        const int of = __shfl_sync(0xffffffffu, ex, d);
        const int v = of == ACT8_NAN ? 0 : act8_quantise(z[d], act8_inverse_step(of));
        if (c0 + d * ACT8_BLOCK < b.K) q[d * ACT8_BLOCK] = static_cast<signed char>(v);
    }
}

// out = dY * act'(z), or out = z where GRAD is false (dY is not read).
template <class T, int ACT, bool GRAD>
__global__ void __launch_bounds__(kThreads)
    read_wide_kernel(Blocks b, Checkpoint c, const T *dY, long long lddy, T *out, long long ldo) {
    constexpr int D = kReadDepth<GRAD>;
    const int sub = threadIdx.x & 3;
    const unsigned first = (blockIdx.x * D) * (kThreads / 4) + (threadIdx.x >> 2);
    uint2 w[D];
    int e[D];
    float dy[D][8];
    unsigned row[D];
    int col[D];
    bool in[D];
#pragma unroll
    for (int d = 0; d < D; ++d) {
        const unsigned u = first + d * (kThreads / 4);
        row[d] = b.per_row.quotient(u);
        col[d] = int(u - row[d] * b.per_row.d) * ACT8_BLOCK + sub * 8;
        in[d] = u < b.units && col[d] < b.K && SG_IN_RANGE(b.holds(row[d], col[d], 8));
        if (!in[d]) continue;
        w[d] = *reinterpret_cast<const uint2 *>(c.q + row[d] * c.ldq + col[d]);
        e[d] = c.e[row[d] * c.lde + col[d] / ACT8_BLOCK];
        if constexpr (GRAD) load8(dY + (long long)row[d] * lddy + col[d], dy[d]);
    }
#pragma unroll
    for (int d = 0; d < D; ++d) {
        if (!in[d]) continue;
        const float step = act8_step(e[d]);
        float z[8];
        unpack_s8(w[d].x, z);
        unpack_s8(w[d].y, z + 4);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            float2 v = __fmul2_rn(make_float2(z[i], z[i + 1]), both(step));
            if constexpr (GRAD) v = __fmul2_rn(make_float2(dy[d][i], dy[d][i + 1]), slope<T, ACT>(v));
            z[i] = v.x, z[i + 1] = v.y;
        }
        store8(out + (long long)row[d] * ldo + col[d], z);
    }
}

template <class T, int ACT, bool GRAD>
__global__ void __launch_bounds__(kThreads, 6)
    read_any_kernel(Blocks b, Checkpoint c, const T *dY, long long lddy, T *out, long long ldo) {
    constexpr int D = kAnyDepth;
    const int lane = threadIdx.x & 31;
    const unsigned u = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), row = b.per_row.quotient(u);
    if (u >= b.units) return;
    const int c0 = int(u - row * b.per_row.d) * (D * ACT8_BLOCK) + lane;
    if (!SG_IN_RANGE(b.holds(row, c0 - lane, 1))) return;
    const signed char *q = c.q + row * c.ldq + c0, *e = c.e + row * c.lde + (c0 - lane) / ACT8_BLOCK;
    const T *dyr = GRAD ? dY + (long long)row * lddy + c0 : nullptr;
    T *to = out + (long long)row * ldo + c0;
    signed char w[D];
    float dy[D];
    const int mine = lane < D && c0 - lane + lane * ACT8_BLOCK < b.K ? e[lane] : 0;
#pragma unroll
    for (int d = 0; d < D; ++d) {
        const bool in = c0 + d * ACT8_BLOCK < b.K;
        w[d] = in ? q[d * ACT8_BLOCK] : 0;
        if constexpr (GRAD) dy[d] = in ? to_f32(dyr[d * ACT8_BLOCK]) : 0.0f;
    }
#pragma unroll
    for (int d = 0; d < D; d += 2) {
        float2 v = make_float2(float(w[d]) * act8_step(__shfl_sync(0xffffffffu, mine, d)),
                               float(w[d + 1]) * act8_step(__shfl_sync(0xffffffffu, mine, d + 1)));
        if constexpr (GRAD) v = __fmul2_rn(make_float2(dy[d], dy[d + 1]), slope<T, ACT>(v));
        if (c0 + d * ACT8_BLOCK < b.K) to[d * ACT8_BLOCK] = from_f32<T>(v.x);
        if (c0 + (d + 1) * ACT8_BLOCK < b.K) to[(d + 1) * ACT8_BLOCK] = from_f32<T>(v.y);
    }
}

// ------------------------------------------------------------------ host
bool aligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// A matrix whose rows of K elements can be read eight at a time.
template <class T>
bool wide(const T *p, int ld) {
    return !p || (aligned(p, sizeof(T) == 1 ? 8 : 16) && ld % 8 == 0);
}

int check_sizes(int type, int M, int K) {
    if (type != SGEMM_F32 && type != SGEMM_BF16) return SGEMM_ERR_INVALID_ARG;
    if (M < 0 || K < 0) return SGEMM_ERR_INVALID_ARG;
    if (M > sgh::kMaxDim || K > sgh::kMaxDim) return SGEMM_ERR_TOO_LARGE;
    return SGEMM_OK;
}
bool bad_matrix(const void *p, int ld, int columns, size_t element) {
    return !p || !aligned(p, element) || ld < std::max(1, columns);
}
size_t element_bytes(int type) { return type == SGEMM_BF16 ? 2 : 4; }
int blocks_of(int K) { return (K + ACT8_BLOCK - 1) / ACT8_BLOCK; }

// Calls launch(first row, rows) for row ranges of fewer than 2^31 blocks, so that
// the kernels number them in 32 bits.
template <class F>
int over_rows(int M, int K, F &&launch) {
    int sms;
    cudaMemPool_t pool;
    const int st = sgh::current_device(&sms, &pool);
    if (st != SGEMM_OK) return st;
    const long long most = std::max<long long>(1, 0x7ff00000LL / blocks_of(K));
    for (long long r = 0; r < M; r += most) {
        launch(r, int(std::min<long long>(most, M - r)));
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return sgh::cuda_fail(e);
    }
    return SGEMM_OK;
}

Blocks blocks_in(int rows, int K, bool wide_form) {
    const unsigned per_row = unsigned(wide_form ? blocks_of(K) : (blocks_of(K) + kAnyDepth - 1) / kAnyDepth);
    return Blocks{unsigned(rows) * per_row, Divisor::of(per_row), K};
}
unsigned grid_of(unsigned units, unsigned per_block) { return (units + per_block - 1) / per_block; }

template <class T, int ACT, bool WITH_Y>
int store(int M, int K, const T *Z, int ldz, Checkpoint c, T *Y, int ldy, cudaStream_t stream) {
    const bool w = K % 8 == 0 && wide(Z, ldz) && wide(Y, ldy) && wide(c.q, int(c.ldq));
    return over_rows(M, K, [&](long long r, int rows) {
        const Blocks b = blocks_in(rows, K, w);
        const Checkpoint at{c.q + r * c.ldq, c.e + r * c.lde, c.ldq, c.lde};
        T *y = WITH_Y ? Y + r * ldy : nullptr;
        if (w)
            store_wide_kernel<T, ACT, WITH_Y>
                <<<grid_of(b.units, kStoreDepth<T> * kThreads / 4), kThreads, 0, stream>>>(
                    b, Z + r * ldz, ldz, at, y, ldy);
        else
            store_any_kernel<T, ACT, WITH_Y>
                <<<grid_of(b.units, kThreads / 32), kThreads, 0, stream>>>(
                    b, Z + r * ldz, ldz, at, y, ldy);
        sgh::count_launch(w ? "act8 store, rows read 16 bytes at a time"
                            : "act8 store, any alignment");
    });
}

template <class T, int ACT, bool GRAD>
int read(int M, int K, Checkpoint c, const T *dY, int lddy, T *out, int ldo, cudaStream_t stream) {
    const bool w = K % 8 == 0 && wide(dY, lddy) && wide(out, ldo) && wide(c.q, int(c.ldq));
    return over_rows(M, K, [&](long long r, int rows) {
        const Blocks b = blocks_in(rows, K, w);
        const Checkpoint at{c.q + r * c.ldq, c.e + r * c.lde, c.ldq, c.lde};
        const T *dy = GRAD ? dY + r * lddy : nullptr;
        if (w)
            read_wide_kernel<T, ACT, GRAD>
                <<<grid_of(b.units, kReadDepth<GRAD> * kThreads / 4), kThreads, 0, stream>>>(
                    b, at, dy, lddy, out + r * ldo, ldo);
        else
            read_any_kernel<T, ACT, GRAD>
                <<<grid_of(b.units, kThreads / 32), kThreads, 0, stream>>>(
                    b, at, dy, lddy, out + r * ldo, ldo);
        sgh::count_launch(w ? "act8 read, rows read 16 bytes at a time"
                            : "act8 read, any alignment");
    });
}

template <class T>
int store_typed(int M, int K, const void *Z, int ldz, int act, Checkpoint c, void *Y, int ldy,
                cudaStream_t s) {
    const T *z = static_cast<const T *>(Z);
    T *y = static_cast<T *>(Y);
    if (!y) return store<T, SGEMM_ACT_NONE, false>(M, K, z, ldz, c, y, 0, s);
    if (act == SGEMM_ACT_RELU) return store<T, SGEMM_ACT_RELU, true>(M, K, z, ldz, c, y, ldy, s);
    if (act == SGEMM_ACT_GELU) return store<T, SGEMM_ACT_GELU, true>(M, K, z, ldz, c, y, ldy, s);
    return store<T, SGEMM_ACT_NONE, true>(M, K, z, ldz, c, y, ldy, s);
}

template <class T>
int grad_typed(int M, int K, Checkpoint c, int act, const void *dY, int lddy, void *dZ, int lddz,
               cudaStream_t s) {
    const T *dy = static_cast<const T *>(dY);
    T *dz = static_cast<T *>(dZ);
    if (act == SGEMM_ACT_RELU) return read<T, SGEMM_ACT_RELU, true>(M, K, c, dy, lddy, dz, lddz, s);
    if (act == SGEMM_ACT_GELU) return read<T, SGEMM_ACT_GELU, true>(M, K, c, dy, lddy, dz, lddz, s);
    return read<T, SGEMM_ACT_NONE, true>(M, K, c, dy, lddy, dz, lddz, s);
}

bool bad_act(int act) { return act < SGEMM_ACT_NONE || act > SGEMM_ACT_GELU; }

// A checkpoint that only is read.
Checkpoint readable(const signed char *q, int ldq, const signed char *e, int lde) {
    return Checkpoint{const_cast<signed char *>(q), const_cast<signed char *>(e), ldq, lde};
}

}  // namespace

cudaError_t sgh::act8_error_word(unsigned *v, bool clear) { return sgv::unit_error_word(v, clear); }

SGEMM_API int sgemm_act8_store(int type, int M, int K, const void *Z, int ldz, int act,
                               signed char *q, int ldq, signed char *e, int lde, void *Y, int ldy,
                               sgemm_stream_t stream) {
    const int st = check_sizes(type, M, K);
    if (st != SGEMM_OK) return st;
    if (bad_act(act)) return SGEMM_ERR_INVALID_ARG;
    if (M == 0 || K == 0) return SGEMM_OK;
    if (bad_matrix(Z, ldz, K, element_bytes(type)) || bad_matrix(q, ldq, K, 1) ||
        bad_matrix(e, lde, blocks_of(K), 1) || (Y && bad_matrix(Y, ldy, K, element_bytes(type))))
        return SGEMM_ERR_INVALID_ARG;
    const Checkpoint c{q, e, ldq, lde};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return type == SGEMM_BF16 ? store_typed<bf16>(M, K, Z, ldz, act, c, Y, ldy, s)
                              : store_typed<float>(M, K, Z, ldz, act, c, Y, ldy, s);
}

SGEMM_API int sgemm_act8_load(int type, int M, int K, const signed char *q, int ldq,
                              const signed char *e, int lde, void *X, int ldx,
                              sgemm_stream_t stream) {
    const int st = check_sizes(type, M, K);
    if (st != SGEMM_OK) return st;
    if (M == 0 || K == 0) return SGEMM_OK;
    if (bad_matrix(X, ldx, K, element_bytes(type)) || bad_matrix(q, ldq, K, 1) ||
        bad_matrix(e, lde, blocks_of(K), 1))
        return SGEMM_ERR_INVALID_ARG;
    const Checkpoint c = readable(q, ldq, e, lde);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return type == SGEMM_BF16
               ? read<bf16, SGEMM_ACT_NONE, false>(M, K, c, nullptr, 0, static_cast<bf16 *>(X), ldx, s)
               : read<float, SGEMM_ACT_NONE, false>(M, K, c, nullptr, 0, static_cast<float *>(X), ldx, s);
}

SGEMM_API int sgemm_act8_grad(int type, int M, int K, const signed char *q, int ldq,
                              const signed char *e, int lde, int act, const void *dY, int lddy,
                              void *dZ, int lddz, sgemm_stream_t stream) {
    const int st = check_sizes(type, M, K);
    if (st != SGEMM_OK) return st;
    if (bad_act(act)) return SGEMM_ERR_INVALID_ARG;
    if (M == 0 || K == 0) return SGEMM_OK;
    if (bad_matrix(dY, lddy, K, element_bytes(type)) || bad_matrix(dZ, lddz, K, element_bytes(type)) ||
        bad_matrix(q, ldq, K, 1) || bad_matrix(e, lde, blocks_of(K), 1))
        return SGEMM_ERR_INVALID_ARG;
    const Checkpoint c = readable(q, ldq, e, lde);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return type == SGEMM_BF16 ? grad_typed<bf16>(M, K, c, act, dY, lddy, dZ, lddz, s)
                              : grad_typed<float>(M, K, c, act, dY, lddy, dZ, lddz, s);
}
