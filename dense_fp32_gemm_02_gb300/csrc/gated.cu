// gated.cu -- entry points of the gated block, forward and backward.
#include "gated_tiles.cuh"
#include "layer_host.h"
#include "packed.cuh"
#include "pair_gemm.h"
#include "split_tiles.cuh"
#include "variant.cuh"

#define SGEMM_API extern "C" __attribute__((visibility("default")))

namespace {

using namespace sgl;

constexpr const char *kFewRows = "gated, few rows, both matrices read once";

struct Call {
    int type, M, N, K, act;
    const void *X;
    int ldx;
    const void *Wg;
    int ldwg;
    const void *Wu;
    int ldwu;
    void *G;
    int ldg;
    void *U;
    int ldu;
    void *H;   // backward: dH
    int ldh;
    void *dX;
    int lddx;
    void *dWg;
    int lddwg;
    void *dWu;
    int lddwu;
    cudaStream_t stream;
};

int zero(void *p, int ld, int rows, int columns, size_t element, cudaStream_t stream) {
    if (!p || rows == 0 || columns == 0) return SGEMM_OK;
    const cudaError_t e = cudaMemset2DAsync(p, size_t(ld) * element, 0, size_t(columns) * element, size_t(rows), stream);
    return e == cudaSuccess ? SGEMM_OK : sgh::cuda_fail(e);
}

// Sums of ranges, `pitch` apart in a range and `plane` from one range to the next.
template <class T, bool GATED>
int finish(int M, int N, int ranges, const float *x, const float *y, long long pitch, long long plane,
           const PairOut<T> &to, cudaStream_t stream) {
    const bool wide = N % 4 == 0 && pitch % 4 == 0 && plane % 4 == 0 && sgh::aligned(x, 16) && sgh::aligned(y, 16);
    return sgh::launch(nullptr, pair_finish_kernel<T, GATED>, dim3(unsigned((N + 511LL) / 512), unsigned(std::min(M, 65535))),
                       128, 0, stream, M, N, ranges, x, y, pitch, plane, wide, to);
}

// The operands that the TMA does not read where they lie, as parts.  `beside`: not the call's first kernel, it
// runs beside the one before it (host_state.h).
template <class T>
int pack(const Packed<T> &Wg, const Packed<T> &Wu, const Packed<T> &X, bool beside, int sms, cudaStream_t stream) {
    const auto g = Wg.job(), u = Wu.job(), x = X.job();
    const long long octets = g.octets() + u.octets() + x.octets();
    if (octets == 0) return SGEMM_OK;
    const unsigned blocks = unsigned(std::min<long long>((octets + 255) / 256, 32LL * sms));
    return sgh::launch(nullptr, gated_parts_kernel<T>, dim3(blocks), 256, 0, stream, g, u, x, beside);
}

// ------------------------------------------------------------------ forward
// Up to 16 float32 rows: by FMAs to 8 (W through registers once), by warp-level MMAs to 16 (rows.cuh).
int forward_few_rows(const Call &c, int sms, cudaMemPool_t pool) {
    const float *Wg = static_cast<const float *>(c.Wg), *Wu = static_cast<const float *>(c.Wu);
    const bool w_wide = wide_rows(Wg, c.ldwg) && wide_rows(Wu, c.ldwu), stream_rows = c.M <= STREAM_ROWS;
    const Rows<float> X{static_cast<const float *>(c.X), c.ldx};
    RowsWork w{};
    w.M = c.M, w.N = c.N, w.K = c.K;
    w.x_wide = sgh::aligned(c.X, 4 * sizeof(float)) && c.ldx % 4 == 0;
    if (stream_rows)
        split_rows(w, 32 * 16 / int(sizeof(float)), RANK_THREADS / 32 * STREAM_DEPTH, STREAM_RANGE,
                   (long long)sms * stream_blocks(c.M), sizeof(float), 2);
    else
        split_rows(w, ROWS_COLS, SLAB, sgh::kMaxDim, 2LL * sms, sizeof(float), 2);
    const long long blocks = 2LL * w.across * w.ranges, one = (long long)w.ranges * c.M * c.N;
    if (blocks > 0x7fffffffLL) return SGEMM_ERR_TOO_LARGE;
    sgh::Workspace ws(pool, c.stream);
    int st = ws.allocate(sgh::Workspace::piece(size_t(one) * 8));
    if (st != SGEMM_OK) return st;
    w.partial = ws.take<float>(size_t(one) * 2);
    if (stream_rows) {
        auto pick = [&](auto wide) {
            constexpr bool W = decltype(wide)::value;
            return c.M <= 1   ? gated_stream_kernel<1, W>
                   : c.M <= 2 ? gated_stream_kernel<2, W>
                   : c.M <= 4 ? gated_stream_kernel<4, W>
                              : gated_stream_kernel<8, W>;
        };
        auto kernel = w_wide ? pick(std::true_type{}) : pick(std::false_type{});
        st = sgh::launch(kFewRows, kernel, dim3(unsigned(blocks)), RANK_THREADS, 0, c.stream, w, X, Wg, (long long)c.ldwg, Wu,
                         (long long)c.ldwu);
    } else {
        const size_t smem = FewRows<1>::SMEM;
        const cudaError_t e = cudaFuncSetAttribute(gated_few_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return sgh::cuda_fail(e);
        st = sgh::launch(kFewRows, gated_few_rows_kernel, dim3(unsigned(blocks)), RANK_THREADS, smem, c.stream, w, X, Wg,
                         (long long)c.ldwg, Wu, (long long)c.ldwu, w_wide);
    }
    if (st != SGEMM_OK) return st;
    const PairOut<float> to{static_cast<float *>(c.G), static_cast<float *>(c.U), static_cast<float *>(c.H), c.ldg, c.ldu, c.ldh, c.act};
    st = finish<float, true>(c.M, c.N, w.ranges, w.partial, w.partial + one, c.N, (long long)c.M * c.N, to, c.stream);
    return st == SGEMM_OK ? ws.release() : st;
}

// Few float32 rows, W split on its way (split_tiles.cuh).
int encode_floats(CUtensorMap *map, const float *p, long long inner, long long outer, long long pitch) {
    const cuuint64_t dims[2] = {cuuint64_t(inner), cuuint64_t(outer)}, strides[1] = {cuuint64_t(pitch) * 4};
    const cuuint32_t box[2] = {SPLIT_COLS, SPLIT_STEP}, steps[2] = {1, 1};
    const CUresult r = sgh::encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float *>(p), dims, strides, box,
                                           steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SGEMM_OK : sgh::driver_fail(int(r));
}

int forward_split(const Call &c, bool wide, int sms, cudaMemPool_t pool) {
    SplitWork w{};
    w.M = c.M, w.N = c.N, w.K = c.K;
    w.across = (c.N + SPLIT_COLS - 1) / SPLIT_COLS;
    w.down = (c.M + SPLIT_ROWS - 1) / SPLIT_ROWS;
    w.rows = ((c.M + w.down - 1) / w.down + 15) / 16 * 16;
    w.timeout_ns = sgh::wait_timeout_ns();
    const int steps = (c.K + SPLIT_STEP - 1) / SPLIT_STEP;
    const long long tiles = 2LL * w.across * w.down, one = (long long)c.M * c.N;
    double least = 0;
    for (int n = 1; n <= std::min(steps, 64); ++n) {   // us: a slab, filling and emptying a block, the ranges' sums
        const int per = (steps + n - 1) / n;
        if ((steps + per - 1) / per != n) continue;   // a range would be empty
        const double cost = double((tiles * n + sms - 1) / sms) * (per * 1.0 + 6.0) + n * double(one) * 16 / 5.0e6;
        if (w.ranges == 0 || cost < least) least = cost, w.ranges = n, w.range = per * SPLIT_STEP;
    }
    if (tiles * w.ranges > 0x7fffffffLL) return SGEMM_ERR_TOO_LARGE;
    Packed<float> X(c.M, c.K, c.X, c.ldx), none(0, 0, nullptr, 8);
    sgh::Workspace ws(pool, c.stream);
    int st = ws.allocate(X.bytes() + sgh::Workspace::piece(size_t(one) * w.ranges * 8));
    if (st != SGEMM_OK) return st;
    X.place(ws);
    w.partial = ws.take<float>(size_t(one) * w.ranges * 2);
    if ((st = pack(none, none, X, false, sms, c.stream)) != SGEMM_OK) return st;
    const SplitWeights weights{{static_cast<const float *>(c.Wg), static_cast<const float *>(c.Wu)}, {c.ldwg, c.ldwu}};
    CUtensorMap mX, mG, mU;
    if ((st = sgp::encode(&mX, X.operand(), SPLIT_STEP, unsigned(w.rows))) != SGEMM_OK) return st;
    mG = mU = mX;
    if (wide && ((st = encode_floats(&mG, weights.p[0], c.N, c.K, c.ldwg)) != SGEMM_OK ||
                 (st = encode_floats(&mU, weights.p[1], c.N, c.K, c.ldwu)) != SGEMM_OK))
        return st;
    const auto kernel = wide ? split_tiles_kernel<true> : split_tiles_kernel<false>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(SPLIT_SMEM));
    if (e != cudaSuccess) return sgh::cuda_fail(e);
    st = sgh::launch("gated, W split into bf16 parts on its way, tcgen05", kernel, dim3(unsigned(tiles * w.ranges)), SPLIT_THREADS,
                     SPLIT_SMEM, c.stream, mX, mG, mU, weights, w);
    if (st != SGEMM_OK) return st;
    const PairOut<float> to{static_cast<float *>(c.G), static_cast<float *>(c.U), static_cast<float *>(c.H), c.ldg, c.ldu, c.ldh, c.act};
    st = finish<float, true>(c.M, c.N, w.ranges, w.partial, w.partial + one * w.ranges, c.N, one, to, c.stream);
    return st == SGEMM_OK ? ws.release() : st;
}

// Float32 rows up to which W is read by warp-level MMAs (rows.cuh), and split on its way to the tensor cores, W's
// rows 16-byte aligned or not; more have its parts laid out first.  us, 16 rows of 4096 x 4096 40.8 by
// warps / 40.7 split, of 704 x 1504 8.0 / 9.7; 192 rows of 4096 x 4096 110 split / 130 laid out, 256 rows 137 / 137 (4096 x
// 8192: 254 / 222).  Not aligned: 17 rows of 2048 x 2047 23.0 by warps / 22.5, 64 rows 37.6 / 25.3, 128 rows 43.3
// laid out / 37.2, 256 rows of 1023 x 3001 36.4 / 65.
constexpr int kWarpRows = 16, kSplitRows = 192, kSplitUnaligned = 128;
// bfloat16 rows whose ranges' sums meet in clusters (gated_tiles.cuh), and not in memory after the pair product.  us, so /
// by the pair product (below three rows: by FMAs): 1 row of 1024 x 1024 4.1 / 6.0, of 4096 x 8192 22.2 / 26.9; 8 rows 4.3 / 8.5
// and 22.7 / 26.5; 64 rows 6.1 / 7.9 and 26.3 / 27.0.  W laid out first: 1 row of 1023 x 3001 11.4 / 12.8 by FMAs, 8 rows
// 11.5 / 17.1, 64 rows 13.6 / 15.6.
constexpr int kTileRows = 64;

// Few bfloat16 rows in one launch (gated_tiles.cuh), after the layout of what the TMA does not read.
int forward_tiles(const Call &c, int sms, cudaMemPool_t pool) {
    GatedTileWork w{};
    w.M = c.M, w.N = c.N, w.K = c.K;
    w.across = (c.N + GATED_COLS - 1) / GATED_COLS;
    w.rows = (c.M + 15) / 16 * 16;
    w.timeout_ns = sgh::wait_timeout_ns();
    const int steps = (c.K + GATED_STEP - 1) / GATED_STEP;
    double least = 0;
    for (int n = 1; n <= std::min(steps, GATED_CLUSTER); ++n) {   // us: a slab, filling and emptying a block, the cluster
        const int per = (steps + n - 1) / n;
        if ((steps + per - 1) / per != n || per * GATED_STEP > GATED_RANGE) continue;   // a range would be empty, or too long
        const double cost = double(((long long)w.across * n + 2 * sms - 1) / (2 * sms)) * (per * 0.5 + 4.0) + 0.25 * n;
        if (w.ranges == 0 || cost < least) least = cost, w.ranges = n, w.range = per * GATED_STEP;
    }
    Packed<bf16> X(c.M, c.K, c.X, c.ldx), Wg(c.K, c.N, c.Wg, c.ldwg), Wu(c.K, c.N, c.Wu, c.ldwu);
    sgh::Workspace ws(pool, c.stream);
    int st;
    if (const size_t bytes = X.bytes() + Wg.bytes() + Wu.bytes()) {
        if ((st = ws.allocate(bytes)) != SGEMM_OK) return st;
        X.place(ws);
        Wg.place(ws);
        Wu.place(ws);
        if ((st = pack(Wg, Wu, X, false, sms, c.stream)) != SGEMM_OK) return st;
    }
    CUtensorMap mX, mG, mU;
    if ((st = sgp::encode(&mX, X.operand(), GATED_STEP, unsigned(w.rows))) != SGEMM_OK ||
        (st = sgp::encode(&mG, Wg.operand(), GATED_STEP, GATED_STEP)) != SGEMM_OK ||
        (st = sgp::encode(&mU, Wu.operand(), GATED_STEP, GATED_STEP)) != SGEMM_OK)
        return st;
    const PairOut<bf16> to{static_cast<bf16 *>(c.G), static_cast<bf16 *>(c.U), static_cast<bf16 *>(c.H), c.ldg, c.ldu, c.ldh, c.act};
    const auto go = [&](auto rows) {
        constexpr int ROWS = decltype(rows)::value;
        const auto kernel = gated_tiles_kernel<ROWS>;
        constexpr size_t smem = GatedTile<ROWS>::SMEM;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return sgh::cuda_fail(e);
        const long long blocks = (long long)w.across * w.ranges;
        return sgh::launch_cluster("gated, few rows, tcgen05, sums in clusters", kernel, dim3(unsigned(blocks)), GATED_THREADS, smem, w.ranges,
                                   c.stream, mX, mG, mU, w, to);
    };
    st = w.rows <= 16   ? go(std::integral_constant<int, 16>{})
         : w.rows <= 32 ? go(std::integral_constant<int, 32>{})
                        : go(std::integral_constant<int, 64>{});
    return st == SGEMM_OK ? ws.release() : st;
}

template <class T>
int forward(const Call &c) {
    int sms, st;
    cudaMemPool_t pool;
    if ((st = sgh::current_device(&sms, &pool)) != SGEMM_OK) return st;
    constexpr int PARTS = Packed<T>::PARTS;
    const PairOut<T> to{static_cast<T *>(c.G), static_cast<T *>(c.U), static_cast<T *>(c.H), c.ldg, c.ldu, c.ldh, c.act};
    if (c.K == 0) return finish<T, true>(c.M, c.N, 0, nullptr, nullptr, c.N, 0, to, c.stream);
    if constexpr (PARTS == 3) {
        if (c.M <= kWarpRows) return forward_few_rows(c, sms, pool);
        const bool wide = wide_rows(static_cast<const T *>(c.Wg), c.ldwg) && wide_rows(static_cast<const T *>(c.Wu), c.ldwu);
        if (c.M <= (wide ? kSplitRows : kSplitUnaligned)) return forward_split(c, wide, sms, pool);
    } else {
        if (c.M <= kTileRows && c.K <= GATED_CLUSTER * GATED_RANGE) return forward_tiles(c, sms, pool);
    }
    Packed<T> X(c.M, c.K, c.X, c.ldx), Wg(c.K, c.N, c.Wg, c.ldwg), Wu(c.K, c.N, c.Wu, c.ldwu);
    const sgp::Split split = sgq::plan(sgq::GATE, c.M, c.N, c.K, PARTS == 3 ? 6 : 1, sms);
    sgh::Workspace ws(pool, c.stream);
    st = ws.allocate(X.bytes() + Wg.bytes() + Wu.bytes() + sgh::Workspace::piece(split.partial_floats * 4));
    if (st != SGEMM_OK) return st;
    X.place(ws);
    Wg.place(ws);
    Wu.place(ws);
    float *partial = split.partial_floats ? ws.take<float>(split.partial_floats) : nullptr;
    if ((st = pack(Wg, Wu, X, false, sms, c.stream)) != SGEMM_OK) return st;
    sgq::Product g{c.M, c.N, c.K, X.operand(), {Wg.operand(), Wu.operand()}};
    const sgq::Output<T> out{to.out, to.out1, to.H, to.ldo, to.ldo1, to.ldh, to.act, nullptr, nullptr, nullptr, nullptr};
    if ((st = sgq::run<T, sgq::GATE>(g, out, split, partial, sms, c.stream)) != SGEMM_OK) return st;
    if (partial) {
        st = finish<T, true>(c.M, c.N, split.splits, partial, partial + c.N, 2LL * c.N, 2LL * c.M * c.N, to, c.stream);
        if (st != SGEMM_OK) return st;
    }
    return ws.release();
}

// ------------------------------------------------------------------ backward
template <class T>
int backward(const Call &c) {
    int sms, st;
    cudaMemPool_t pool;
    if ((st = sgh::current_device(&sms, &pool)) != SGEMM_OK) return st;
    constexpr int PARTS = Packed<T>::PARTS, PRODUCTS = PARTS == 3 ? 6 : 1;
    const bool want_dx = c.dX != nullptr, want_dw = c.dWg != nullptr;
    Packed<T> X(c.M, c.K, c.X, c.ldx), Wg(c.K, c.N, c.Wg, c.ldwg), Wu(c.K, c.N, c.Wu, c.ldwu);
    if (!want_dw) X.direct = true;                  // no parts of them are needed
    if (!want_dx) Wg.direct = Wu.direct = true;
    const sgp::Split sum = want_dx ? sgq::plan(sgq::SUM, c.M, c.K, c.N, PRODUCTS, sms) : sgp::Split{1, 256, 0};
    const sgp::Split two = want_dw ? sgq::plan(sgq::TWO, c.K, c.N, c.M, PRODUCTS, sms) : sgp::Split{1, 256, 0};
    const long long pitch = pitch8(c.N), plane = c.M * pitch;
    const size_t d_elems = size_t(2) * PARTS * plane;
    sgh::Workspace ws(pool, c.stream);
    st = ws.allocate(sgh::Workspace::piece(d_elems * 2) + X.bytes() + Wg.bytes() + Wu.bytes() +
                     sgh::Workspace::piece(sum.partial_floats * 4) + sgh::Workspace::piece(two.partial_floats * 4));
    if (st != SGEMM_OK) return st;
    bf16 *d = ws.take<bf16>(d_elems);
    X.place(ws);
    Wg.place(ws);
    Wu.place(ws);
    float *sum_partial = sum.partial_floats ? ws.take<float>(sum.partial_floats) : nullptr;
    float *two_partial = two.partial_floats ? ws.take<float>(two.partial_floats) : nullptr;

    SlopesJob<T> job{static_cast<const T *>(c.H), static_cast<const T *>(c.G), static_cast<const T *>(c.U), c.ldh, c.ldg, c.ldu,
                     c.M, c.N, c.act, false, {d, pitch, plane}, {d + PARTS * plane, pitch, plane},
                     Divisor::of(unsigned((c.N + 7LL) / 8))};
    job.wide = wide_rows(job.dH, job.ldh) && wide_rows(job.G, job.ldg) && wide_rows(job.U, job.ldu);
    const long long octets = (long long)c.M * job.per_row.d;
    st = sgh::launch(nullptr, gated_slopes_kernel<T>, dim3(unsigned(std::min<long long>((octets + 255) / 256, 32LL * sms))), 256,
                     0, c.stream, job);
    if (st != SGEMM_OK || (st = pack(Wg, Wu, X, true, sms, c.stream)) != SGEMM_OK) return st;
    const sgp::Operand dG{d, c.N, c.M, PARTS, pitch, plane}, dU{d + PARTS * plane, c.N, c.M, PARTS, pitch, plane};
    if (want_dx) {
        sgq::Product g{c.M, c.K, c.N, {d, c.N, c.M, 2 * PARTS, pitch, plane}, {Wg.operand(), Wu.operand()}};
        const sgq::Output<T> out{static_cast<T *>(c.dX), nullptr, nullptr, c.lddx, 0, 0, 0, nullptr, nullptr, nullptr, nullptr};
        if ((st = sgq::run<T, sgq::SUM>(g, out, sum, sum_partial, sms, c.stream)) != SGEMM_OK) return st;
        if (sum_partial) {
            const sgp::Epilogue<T, false> epi{Adapters{}, nullptr, 0, {}, nullptr, 0.0f, out.out, out.ldo};
            st = sgp::finish<T, false>(c.M, c.K, sum.splits, sum_partial, nullptr, epi, c.stream);
            if (st != SGEMM_OK) return st;
        }
    }
    if (want_dw) {
        sgq::Product g{c.K, c.N, c.M, X.operand(), {dG, dU}};
        const PairOut<T> to{static_cast<T *>(c.dWg), static_cast<T *>(c.dWu), nullptr, c.lddwg, c.lddwu, 0, 0};
        const sgq::Output<T> out{to.out, to.out1, nullptr, to.ldo, to.ldo1, 0, 0, nullptr, nullptr, nullptr, nullptr};
        if ((st = sgq::run<T, sgq::TWO>(g, out, two, two_partial, sms, c.stream)) != SGEMM_OK) return st;
        if (two_partial) {
            st = finish<T, false>(c.K, c.N, two.splits, two_partial, two_partial + c.N, 2LL * c.N, 2LL * c.K * c.N, to,
                                  c.stream);
            if (st != SGEMM_OK) return st;
        }
    }
    return ws.release();
}

}  // namespace

cudaError_t sgh::gated_error_word(unsigned *v, bool clear) { return sgv::unit_error_word(v, clear); }

SGEMM_API int sgemm_gated(int type, int M, int N, int K, const void *X, int ldx, const void *Wg, int ldwg, const void *Wu,
                          int ldwu, int act, void *G, int ldg, void *U, int ldu, void *H, int ldh, sgemm_stream_t stream) {
    const int st = sgh::check_sizes(type, {M, N, K});
    if (st != SGEMM_OK) return st;
    if (act < SGEMM_ACT_NONE || act > SGEMM_ACT_SILU) return SGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return SGEMM_OK;
    const size_t size = sgh::element_bytes(type);
    if ((K > 0 && (sgh::bad_matrix(X, ldx, K, size) || sgh::bad_matrix(Wg, ldwg, N, size) || sgh::bad_matrix(Wu, ldwu, N, size))) ||
        !G != !U || sgh::bad_optional(G, ldg, N, size) || sgh::bad_optional(U, ldu, N, size) || sgh::bad_matrix(H, ldh, N, size))
        return SGEMM_ERR_INVALID_ARG;
    Call c{};
    c.type = type, c.M = M, c.N = N, c.K = K, c.act = act;
    c.X = X, c.ldx = ldx, c.Wg = Wg, c.ldwg = ldwg, c.Wu = Wu, c.ldwu = ldwu;
    c.G = G, c.ldg = ldg, c.U = U, c.ldu = ldu, c.H = H, c.ldh = ldh;
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    return type == SGEMM_BF16 ? forward<bf16>(c) : forward<float>(c);
}

SGEMM_API int sgemm_gated_backward(int type, int M, int N, int K, int act, const void *dH, int lddh, const void *X, int ldx,
                                   const void *G, int ldg, const void *U, int ldu, const void *Wg, int ldwg, const void *Wu,
                                   int ldwu, void *dX, int lddx, void *dWg, int lddwg, void *dWu, int lddwu,
                                   sgemm_stream_t stream) {
    int st = sgh::check_sizes(type, {M, N, K});
    if (st != SGEMM_OK) return st;
    if (act < SGEMM_ACT_NONE || act > SGEMM_ACT_SILU) return SGEMM_ERR_INVALID_ARG;
    const size_t size = sgh::element_bytes(type);
    const bool want_dx = dX && M > 0 && K > 0, want_dw = (dWg || dWu) && K > 0 && N > 0;
    if (want_dw && (!dWg || !dWu || sgh::bad_matrix(dWg, lddwg, N, size) || sgh::bad_matrix(dWu, lddwu, N, size)))
        return SGEMM_ERR_INVALID_ARG;
    if (want_dx && (sgh::bad_matrix(dX, lddx, K, size) ||
                    (N > 0 && (sgh::bad_matrix(Wg, ldwg, N, size) || sgh::bad_matrix(Wu, ldwu, N, size)))))
        return SGEMM_ERR_INVALID_ARG;
    if ((want_dx || want_dw) && M > 0 && N > 0 &&
        (sgh::bad_matrix(dH, lddh, N, size) || sgh::bad_matrix(G, ldg, N, size) || sgh::bad_matrix(U, ldu, N, size)))
        return SGEMM_ERR_INVALID_ARG;
    if (want_dw && M > 0 && sgh::bad_matrix(X, ldx, K, size)) return SGEMM_ERR_INVALID_ARG;
    if (!want_dx && !want_dw) return SGEMM_OK;
    Call c{};
    c.type = type, c.M = M, c.N = N, c.K = K, c.act = act;
    c.H = const_cast<void *>(dH), c.ldh = lddh, c.X = X, c.ldx = ldx;
    c.G = const_cast<void *>(G), c.ldg = ldg, c.U = const_cast<void *>(U), c.ldu = ldu;
    c.Wg = Wg, c.ldwg = ldwg, c.Wu = Wu, c.ldwu = ldwu;
    c.dX = want_dx ? dX : nullptr, c.lddx = lddx;
    c.dWg = want_dw ? dWg : nullptr, c.lddwg = lddwg, c.dWu = want_dw ? dWu : nullptr, c.lddwu = lddwu;
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    if (M == 0 || N == 0) {   // sums of nothing
        int sms;
        cudaMemPool_t pool;
        if ((st = sgh::current_device(&sms, &pool)) != SGEMM_OK) return st;
        if ((st = zero(c.dX, lddx, M, K, size, c.stream)) != SGEMM_OK || (st = zero(c.dWg, lddwg, K, N, size, c.stream)) != SGEMM_OK)
            return st;
        return zero(c.dWu, lddwu, K, N, size, c.stream);
    }
    return type == SGEMM_BF16 ? backward<bf16>(c) : backward<float>(c);
}
