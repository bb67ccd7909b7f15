// lora.cu -- entry points of the adapter layer and of the weight gradient from an
// 8-bit checkpoint: argument checks, workspaces and launches.
#include <algorithm>

#include "../../include/sgemm_layers.h"
#include "host_state.h"
#include "packed.cuh"
#include "parts_gemm.h"
#include "rank_products.cuh"
#include "rows.cuh"
#include "variant.cuh"

#define SGEMM_API extern "C" __attribute__((visibility("default")))

namespace {

using namespace sgl;
using sgh::aligned;

constexpr int kMaxRank = 128, kMaxAdapters = 1024;

bool bad_matrix(const void *p, int ld, int columns, size_t element) {
    return !p || !aligned(p, element) || ld < std::max(1, columns);
}
size_t element_bytes(int type) { return type == SGEMM_BF16 ? 2 : 4; }
int blocks_of(int K) { return (K + ACT8_BLOCK - 1) / ACT8_BLOCK; }

int launched(const char *main_kernel = nullptr) {
    sgh::count_launch(main_kernel);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SGEMM_OK : sgh::cuda_fail(e);
}

// One call of the adapter layer, forward or backward (what a direction does not
// have is null).
struct Call {
    int type, M, N, K, L, R;
    const void *X;
    int ldx;
    const signed char *q;
    int ldq;
    const signed char *e;
    int lde;
    const void *W;
    int ldw;
    const void *A;
    int lda;
    long long stride_a;
    const void *B;
    int ldb;
    long long stride_b;
    const int *ids, *ranks;
    const float *scales;
    const void *bias;
    float *H;
    int ldh;
    void *Y;
    int ldy;
    const void *dY;
    int lddy;
    void *dX;
    int lddx;
    void *dA;
    int ldda;
    long long stride_da;
    void *dB;
    int lddb;
    long long stride_db;
    cudaStream_t stream;

    Adapters adapters() const { return Adapters{ids, ranks, scales, L, R}; }
};

int check_sizes(int type, int M, int N, int K) {
    if (type != SGEMM_F32 && type != SGEMM_BF16) return SGEMM_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 0) return SGEMM_ERR_INVALID_ARG;
    if (M > sgh::kMaxDim || N > sgh::kMaxDim || K > sgh::kMaxDim) return SGEMM_ERR_TOO_LARGE;
    return SGEMM_OK;
}

// Sizes, and the stack's shape, ids, ranks and scales.
int check_common(const Call &c) {
    const int st = check_sizes(c.type, c.M, c.N, c.K);
    if (st != SGEMM_OK) return st;
    if (c.L < 0 || c.L > kMaxAdapters || (c.L > 0 && (c.R < 1 || c.R > kMaxRank)))
        return SGEMM_ERR_INVALID_ARG;
    if (c.L > 0 && ((c.M > 0 && !c.ids) || !aligned(c.ids, 4) || !aligned(c.ranks, 4) ||
                    !aligned(c.scales, 4)))
        return SGEMM_ERR_INVALID_ARG;
    return SGEMM_OK;
}
// A stack of L matrices of rows x columns.
bool bad_stack(const void *p, int ld, long long stride, int L, int rows, int columns, size_t element) {
    if (rows == 0 || columns == 0) return false;
    return bad_matrix(p, ld, columns, element) ||
           (L > 1 && stride < (long long)(rows - 1) * ld + columns);
}

// ------------------------------------------------------------------ operands
template <class T>
Stack<const T> stack_of(const void *p, int ld, long long stride) {
    return {static_cast<const T *>(p), ld, stride};
}
template <class T>
bool wide_stack(const Stack<T> &v, int L) {
    return wide_rows(v.p, v.ld) && (L <= 1 || v.stride % (16 / (long long)sizeof(T)) == 0);
}

// Raises a kernel's shared memory limit; on every launch, as it costs less than
// remembering the devices it was done on.  `bytes` is the same in every call for a kernel.
constexpr size_t DEFAULT_SHARED = 40 * 1024;   // (48 KB less what a kernel declares itself)
template <class K>
int shared_limit(K kernel, size_t bytes) {
    if (bytes <= DEFAULT_SHARED) return SGEMM_OK;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
    return e == cudaSuccess ? SGEMM_OK : sgh::cuda_fail(e);
}

// A launch after current_device(): early (host_state.h), counted, its errors returned.
template <class... P, class... Args>
int launch(const char *text, void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
           const Args &...args) {
    const cudaError_t e = sgh::launch_early(kernel, grid, threads, smem, stream, args...);
    return e == cudaSuccess ? launched(text) : sgh::cuda_fail(e);
}

// ------------------------------------------------------------------ the first kernels
// Lays the planes out (g.planes not null), sorts the rows by adapter (g.perm not null) and
// takes the operands' parts.
template <int P_PARTS, int Q_PARTS, class XP, class XQ>
int prepare(int M, const Adapters &ad, const Groups &g, const PartsJob<XP> &p, const PartsJob<XQ> &q, int sms,
            cudaStream_t stream) {
    int st = SGEMM_OK;
    if (g.planes) {
        // (the limit is the process's: never this call's size, which another thread's may exceed)
        if (sort_smem(ad.L) > DEFAULT_SHARED && (st = shared_limit(group_rows_kernel, sort_smem(kMaxAdapters))) != SGEMM_OK)
            return st;
        st = launch(nullptr, group_rows_kernel, dim3(g.perm ? 2 : 1), SORT_THREADS, sort_smem(ad.L), stream, M, ad, g);
        if (st != SGEMM_OK) return st;
    }
    const long long octets = p.octets() + q.octets();
    if (octets == 0) return SGEMM_OK;
    const unsigned blocks = unsigned(std::min<long long>((octets + 255) / 256, 32LL * sms));
    return launch(nullptr, parts_kernel<P_PARTS, Q_PARTS, XP, XQ>, dim3(blocks), 256, 0, stream, p, q, g.planes != nullptr);
}

// Sizes and workspace of the grouping of a call's rows.
struct Grouping {
    int M, L, chunk, max_chunks, tiles256, width, most_planes, capacity;
    bool sorted;   // for the stack's gradients
    Groups g{};

    // chunk: rows of a partial sum of the stack's gradients, 512 where that makes
    // blocks for every SM twice, else down to 128 (`columns`: of both gradients, 0: none).
    Grouping(const Call &c, long long columns, int sms) : M(c.M), L(c.L), chunk(CHUNK_ROWS), sorted(columns > 0) {
        const long long across = (columns + 127) / 128;
        while (chunk > 128 && (M / chunk) * across < 2LL * sms) chunk /= 2;
        max_chunks = M / chunk + L;
        tiles256 = (M + 255) / 256;
        // planes: for every adapter in every tile, but at most 512 MB a part
        width = c.R <= 16 ? 16 : c.R <= 32 ? 32 : c.R <= 64 ? 64 : 128;
        most_planes = (std::min(L, std::min(M, 256)) * width + 63) / 64;
        capacity = int(std::min<long long>(16384, (long long)tiles256 * most_planes));
    }
    size_t bytes() const {
        const auto piece = [](size_t n) { return sgh::Workspace::piece(n); };
        return L == 0 ? 0
                      : (sorted ? piece(size_t(M) * 4) + piece(size_t(max_chunks) * 16) + piece(size_t(L + 1) * 4) : 0) +
                            piece(size_t(M) * 4) + 2 * piece(size_t(L) * 4) + piece(size_t(tiles256) * 16) +
                            piece(size_t(tiles256) * most_planes * 16);
    }
    void place(sgh::Workspace &ws) {
        if (L == 0) return;
        if (sorted) {
            g.perm = ws.take<int>(M);
            g.chunks = ws.take<int4>(max_chunks);
            g.chunk_begin = ws.take<int>(L + 1);
            g.max_chunks = max_chunks, g.chunk = chunk;
        }
        g.used = ws.take<int>(L);
        g.unclean = ws.take<int>(L);
        g.planes = ws.take<int4>(tiles256);
        g.plane_adapter = ws.take<int4>(size_t(tiles256) * most_planes);
        g.position = ws.take<int>(M);
        g.most_planes = most_planes, g.capacity = capacity, g.width = width;
    }
};

// ------------------------------------------------------------------ stack gradients
template <class XA, class XB>
struct StackKernel {
    void (*kernel)(StackWork<XA>, StackWork<XB>, int, int, Adapters, Groups);
    size_t smem;

    template <int NT>
    static constexpr StackKernel of() {
        constexpr size_t a = StackTile<XA, NT>::SMEM, b = StackTile<XB, NT>::SMEM;
        return {&stack_tile_kernel<XA, XB, NT>, a > b ? a : b};
    }
    static constexpr StackKernel pick(int R) {
        return R <= 16 ? of<2>() : R <= 32 ? of<4>() : R <= 64 ? of<8>() : of<16>();
    }
};

// dA and dB from X's rows (or their checkpoint's) and dY's, and the parts of G and H.
template <class T, class XA, class XB>
int stack_gradients(const Call &c, const Grouping &gr, XA x, bool x_wide, XB dy, bool dy_wide, const bf16 *s_rows,
                    const bf16 *h_rows, int pitch, float *partial_a, float *partial_b, int sms) {
    const Adapters ad = c.adapters();
    int st;
    if (c.M > 0) {
        const auto k = StackKernel<XA, XB>::pick(c.R);
        if ((st = shared_limit(k.kernel, k.smem)) != SGEMM_OK) return st;
        const StackWork<XA> wa{c.K, x, x_wide, s_rows, partial_a};
        const StackWork<XB> wb{c.N, dy, dy_wide, h_rows, partial_b};
        const long long blocks = ((c.K + 127LL) / 128 + (c.N + 127LL) / 128) * gr.max_chunks;
        if (blocks > 0x7fffffffLL) return SGEMM_ERR_TOO_LARGE;
        st = launch("lora backward, rows grouped by adapter", k.kernel, dim3(unsigned(blocks)), RANK_THREADS, k.smem,
                    c.stream, wa, wb, c.M, pitch, ad, gr.g);
        if (st != SGEMM_OK) return st;
    }
    const long long plane = ((long long)c.K + c.N) * c.R;
    const dim3 grid(unsigned(std::min<long long>((plane + 255) / 256, sms * 8LL)), unsigned(c.L));
    return launch(nullptr, stack_finish_kernel<T>, grid, 256, 0, c.stream, c.K, c.N, ad, (const float *)partial_a,
                  (const float *)partial_b, gr.g, Stack<T>{static_cast<T *>(c.dA), c.ldda, c.stride_da},
                  Stack<T>{static_cast<T *>(c.dB), c.lddb, c.stride_db});
}

// ------------------------------------------------------------------ many rows
// Forward: Y = X W + bias + rank side, S = scale X A.  Backward: dX = dY W^T + G A^T with
// G = scale dY B^T, and the stack's gradients.  In either, with P (X or dY), V1 (A or B^T)
// and V2 (B or A^T): group the rows and take P's and W's parts; S = P V1 and V2's layout;
// S into its planes; P W + S V2 on the tensor cores.
template <class T, bool BACK>
int many_rows(const Call &c, int sms, cudaMemPool_t pool) {
    int st;
    const Adapters ad = c.adapters();
    const int M = c.M, N = BACK ? c.K : c.N, K = BACK ? c.N : c.K;
    void *out = BACK ? c.dX : c.Y;
    const bool ranked = c.L > 0, want_out = out && N > 0 && M > 0, product = want_out && K > 0;
    const bool planes = ranked && product, want_stack = BACK && ranked && (c.dA || c.dB);
    constexpr auto LAYOUT = BACK ? sgp::INPUT_GRAD : sgp::FORWARD;
    constexpr int PRODUCTS = sizeof(T) == 4 ? 6 : 1, PARTS = Packed<T>::PARTS;
    Packed<T> P(M, K, BACK ? c.dY : c.X, BACK ? c.lddy : c.ldx), Q(c.K, c.N, c.W, c.ldw);
    if (!product) Q.direct = true;               // no parts of W are needed,
    if (!product && !ranked) P.direct = true;    // nor of P
    if (M == 0 || K == 0) P.direct = true;       // (nothing of P is read)
    const sgp::Split split = product ? sgp::plan_split(M, N, K, PRODUCTS, sms) : sgp::Split{0, 0, 0};
    Grouping gr(c, want_stack ? (long long)c.K + c.N : 0, sms);
    const int ranges = K > 0 ? sgp::rank_splits(M, K, sms) : 0;   // (no contraction: no sums)
    const int pitch = gr.width;   // of the rows of S and H, as parts
    const long long vpitch = pitch8(N), vplane = gr.width * vpitch, upitch = pitch8(K), uplane = gr.width * upitch;

    sgh::Workspace ws(pool, c.stream);
    const auto piece = [](size_t n) { return sgh::Workspace::piece(n); };
    const size_t s_floats = ranked ? size_t(M) * c.R : 0, r_floats = ranked ? size_t(ranges) * M * gr.width : 0;
    const size_t h_elems = planes ? size_t(S_PARTS) * gr.capacity * 256 * 64 : 0;
    const size_t v_elems = planes ? size_t(PARTS) * c.L * vplane : 0;
    const size_t u_elems = ranked && K > 0 ? size_t(PARTS) * c.L * uplane : 0;
    const size_t row_elems = want_stack ? size_t(S_PARTS) * M * pitch : 0;
    const size_t pa_floats = want_stack ? size_t(gr.max_chunks) * c.R * c.K : 0;
    const size_t pb_floats = want_stack ? size_t(gr.max_chunks) * c.R * c.N : 0;
    st = ws.allocate(gr.bytes() + piece(s_floats * 4) + piece(r_floats * 4) + piece(h_elems * 2) + piece(v_elems * 2) +
                     piece(u_elems * 2) + 2 * piece(row_elems * 2) + piece(pa_floats * 4) + piece(pb_floats * 4) +
                     P.bytes() + Q.bytes() + piece(split.partial_floats * 4));
    if (st != SGEMM_OK) return st;
    gr.place(ws);
    RankSide side{ws.take<float>(s_floats), c.H, c.ldh, nullptr, nullptr, nullptr, pitch, PARTS == 1};
    float *r_partial = ws.take<float>(r_floats);
    const Stack<const T> A = stack_of<T>(c.A, c.lda, c.stride_a), B = stack_of<T>(c.B, c.ldb, c.stride_b);
    const Parts u{ws.take<bf16>(u_elems), upitch, uplane}, v{ws.take<bf16>(v_elems), vpitch, vplane};
    if (planes) side.planes = ws.take<bf16>(h_elems);
    if (want_stack) {
        side.s_rows = ws.take<bf16>(row_elems);
        side.h_rows = ws.take<bf16>(row_elems);
    } else if (BACK) {
        side.H = nullptr;
    }
    float *pa = ws.take<float>(pa_floats), *pb = ws.take<float>(pb_floats);
    P.place(ws);
    Q.place(ws);
    float *partial = split.partial_floats ? ws.take<float>(split.partial_floats) : nullptr;

    st = prepare<PARTS, PARTS>(M, ad, gr.g, P.job(), Q.job(), sms, c.stream);
    if (st != SGEMM_OK) return st;
    if (ranked && M > 0) {
        // V1 with the contraction along its rows, V2 as the product reads it
        const StackSide<T> v1{BACK ? B : A, K, !BACK, false, u}, v2{BACK ? A : B, planes ? N : 0, BACK, true, v};
        const int across = (K + 255) / 256;
        const dim3 grid(unsigned(across + (v2.cols + 255) / 256), unsigned(c.L), unsigned(gr.width / 8));
        if (grid.x > 0) {
            st = launch(nullptr, pack_stack_kernel<T>, grid, 256, 0, c.stream, v1, v2, across, ad, gr.g);
            if (st != SGEMM_OK) return st;
        }
        if (K > 0) {
            const sgp::RankProduct r{M, K, gr.width, gr.most_planes, P.operand(),
                                     {u.p, K, gr.width, (long long)PARTS * c.L, upitch, uplane},
                                     ad, gr.g.planes, gr.g.plane_adapter, gr.g.position};
            if ((st = sgp::run_rank<T>(r, ranges, r_partial, sms, c.stream)) != SGEMM_OK) return st;
        }
        // Four warps to a row where there are few (154 rows of rank 122: 18 -> 6 us; 512 rows
        // of 32 adapters of rank 16: 17 -> 9), else one (8192 rows of rank 64: 7 us, four 15).
        const bool four = M <= 2048;
        st = launch(nullptr, four ? rank_finish_kernel<4> : rank_finish_kernel<1>,
                    dim3(unsigned(four ? (M + 1LL) / 2 : (M + 7LL) / 8)), 256, 0, c.stream, M, ranges,
                    (const float *)r_partial, (long long)M * gr.width, ad, gr.g, side);
        if (st != SGEMM_OK) return st;
    }
    if (want_out) {
        const sgp::Epilogue<T, BACK> epi{ad, side.S, c.R, BACK ? A : B, BACK ? nullptr : static_cast<const T *>(c.bias),
                                         0.0f, static_cast<T *>(out), BACK ? c.lddx : c.ldy};
        if (product) {
            sgp::Product g;
            g.M = M, g.N = N, g.K = K;
            g.a = P.operand();
            g.b = Q.operand();
            if (planes) {
                g.h = {side.planes, 64, 256, (long long)S_PARTS * gr.capacity, 64, 256 * 64};
                g.v = {v.p, N, gr.width, (long long)PARTS * c.L, vpitch, vplane};
                g.planes = gr.g.planes;
                g.plane_adapter = gr.g.plane_adapter;
                g.most_planes = gr.most_planes;
                g.capacity = gr.capacity;
                g.width = gr.width;
            }
            st = sgp::run<T, LAYOUT>(g, epi, split, partial, sms, c.stream);
        } else {   // K == 0: the epilogue of a zero sum
            st = sgp::finish<T, BACK>(M, N, 0, nullptr, nullptr, epi, c.stream);
        }
        if (st != SGEMM_OK) return st;
    }
    if constexpr (BACK) {
        if (want_stack) {
            const Rows<T> x{static_cast<const T *>(c.X), c.ldx};
            const Act8Rows kept{c.q, c.e, c.ldq, c.lde};
            const bool q_wide = aligned(c.q, 16) && c.ldq % 16 == 0, x_wide = wide_rows(x.p, x.ld);
            auto gradients = [&](auto dy, bool dy_wide) {
                return c.X ? stack_gradients<T>(c, gr, x, x_wide, dy, dy_wide, side.s_rows, side.h_rows, pitch, pa, pb, sms)
                           : stack_gradients<T>(c, gr, kept, q_wide, dy, dy_wide, side.s_rows, side.h_rows, pitch, pa, pb, sms);
            };
            if constexpr (sizeof(T) == 4)
                st = gradients(PartRows{P.parts.p, P.pitch, P.parts.plane}, true);
            else
                st = gradients(Rows<T>{P.src, P.ld}, wide_rows(P.src, P.ld));
            if (st != SGEMM_OK) return st;
        }
    }
    return ws.release();
}

// ------------------------------------------------------------------ few rows
constexpr const char *kFewRows = "few rows, W read once, k split over the grid";

template <class T>
using StreamKernel = void (*)(RowsWork, Rows<T>, const T *, long long, Stack<const T>, Adapters);

template <class T, bool WIDE>
StreamKernel<T> stream_kernel(int M) {
    return M <= 1   ? stream_rows_kernel<T, 1, WIDE>
           : M <= 2 ? stream_rows_kernel<T, 2, WIDE>
           : M <= 4 ? stream_rows_kernel<T, 4, WIDE>
                    : stream_rows_kernel<T, 8, WIDE>;
}

// Whether W goes through registers and FMAs.  Of up to 8 rows all do in float32 (8 x 8192 x
// 8192 69 us, the warp-level MMA 77), and bfloat16 until the FMAs of several rows take longer
// than W's bytes: us, by FMAs / by parts_gemm (where W needs no copy), 2 rows 8192 x 8192 30 / 36;
// 4 rows 4096 x 4096 14.3 / 14.8, 4096 x 8192 24.6 / 23.5, 8192 x 8192 44 / 37; 8 rows 2048 x
// 2048 10.7 / 11.4, 3000 x 3000 15.3 / 14.4, 4096 x 4096 19.2 / 15.9, 8192 x 8192 76 / 31.
bool streamed(int M, int K, int N, bool always) {
    if (M > STREAM_ROWS) return false;
    return always || M <= 2 || (long long)K * N < (M <= 4 ? 32000000 : 9000000);
}

// A forward call of few rows: see rows.cuh.
template <class T>
int forward_few_rows(const Call &c, int sms, cudaMemPool_t pool) {
    constexpr bool F32 = sizeof(T) == 4;
    Packed<T> P(c.M, c.K, c.X, c.ldx), Q(c.K, c.N, c.W, c.ldw);   // (of the third kernel)
    const bool stream_rows = streamed(c.M, c.K, c.N, F32 || !Q.direct);
    const bool mma_rows = F32 && !stream_rows && c.M <= MMA_ROWS, ranked = c.L > 0;
    const T *W = static_cast<const T *>(c.W);
    const bool w_wide = wide_rows(W, c.ldw);
    const Adapters ad = c.adapters();
    const Rows<T> X{static_cast<const T *>(c.X), c.ldx};
    const Stack<const T> A = stack_of<T>(c.A, c.lda, c.stride_a), B = stack_of<T>(c.B, c.ldb, c.stride_b);
    int st;
    RowsWork w{};
    w.M = c.M, w.N = c.N, w.K = c.K;
    w.x_wide = aligned(c.X, 4 * sizeof(T)) && c.ldx % 4 == 0;
    w.v_wide = wide_stack(A, c.L);
    sgp::Split split{1, 256, 0};
    auto stream = w_wide ? stream_kernel<T, true>(c.M) : stream_kernel<T, false>(c.M);
    long long slots = sms;
    if (stream_rows) {
        slots *= stream_blocks(c.M);
        split_rows(w, 32 * 16 / int(sizeof(T)), RANK_THREADS / 32 * STREAM_DEPTH, STREAM_RANGE, slots, sizeof(T));
    } else if (mma_rows) {
        slots *= 2;
        split_rows(w, ROWS_COLS, SLAB, sgh::kMaxDim, slots, sizeof(T));
    } else {
        split = sgp::plan_split(c.M, c.N, c.K, F32 ? 6 : 1, sms);
        w.ranges = split.splits;
    }
    if (ranked) {
        const int n = std::max(1, (c.K + 511) / 512);
        w.rank_range = (c.K + n - 1) / n;
        w.rank_ranges = (c.K + w.rank_range - 1) / w.rank_range;
    }
    const size_t p_floats = size_t(w.ranges) * c.M * c.N, r_floats = size_t(w.rank_ranges) * c.M * c.R;
    const bool third = !stream_rows && !mma_rows;
    sgh::Workspace ws(pool, c.stream);
    st = ws.allocate(sgh::Workspace::piece(p_floats * 4) + sgh::Workspace::piece(r_floats * 4) +
                     (third ? P.bytes() + Q.bytes() : 0));
    if (st != SGEMM_OK) return st;
    w.partial = ws.take<float>(p_floats);
    w.rank_partial = ws.take<float>(r_floats);
    const long long product = (long long)w.across * w.ranges, rank = (long long)c.M * w.rank_ranges;
    if (product + rank > 0x7fffffffLL) return SGEMM_ERR_TOO_LARGE;
    const bool together = stream_rows && product + rank <= slots;
    if (third) {
        P.place(ws);
        Q.place(ws);
        st = prepare<Packed<T>::PARTS, Packed<T>::PARTS>(c.M, ad, Groups{}, P.job(), Q.job(), sms, c.stream);
        if (st != SGEMM_OK) return st;
    }
    if (stream_rows) {
        const dim3 grid(unsigned(product + (together ? rank : 0)));
        stream<<<grid, RANK_THREADS, 0, c.stream>>>(w, X, W, c.ldw, A, ad);
        st = launched(kFewRows);
    } else if (mma_rows) {
        if constexpr (F32) {
            auto kernel = c.M <= 16 ? few_rows_kernel<1> : c.M <= 32 ? few_rows_kernel<2> : few_rows_kernel<4>;
            const size_t smem = c.M <= 16 ? FewRows<1>::SMEM : c.M <= 32 ? FewRows<2>::SMEM : FewRows<4>::SMEM;
            if ((st = shared_limit(kernel, smem)) != SGEMM_OK) return st;
            kernel<<<unsigned(product), RANK_THREADS, smem, c.stream>>>(w, X, W, c.ldw, w_wide);
            st = launched(kFewRows);
        }
    } else {
        sgp::Product g;
        g.M = c.M, g.N = c.N, g.K = c.K;
        g.a = P.operand();
        g.b = Q.operand();
        st = sgp::run<T, sgp::FORWARD>(g, sgp::Epilogue<T, false>{}, split, w.partial, sms, c.stream, sgp::PARTIALS);
    }
    if (st != SGEMM_OK) return st;
    if (ranked && !together) {   // it reads nothing of the product's and runs beside it
        const cudaError_t e = sgh::launch_early(few_rows_rank_kernel<T>, dim3(unsigned(rank)), RANK_THREADS, 0, c.stream, w,
                                                X, A, ad);
        if (e != cudaSuccess) return sgh::cuda_fail(e);
        if ((st = launched()) != SGEMM_OK) return st;
    }
    const T *bias = static_cast<const T *>(c.bias);
    const bool wide = (!bias || aligned(bias, 16)) && wide_stack(B, c.L);
    const dim3 grid(unsigned((c.N + 255) / 256), unsigned(c.M));
    const bool early = (long long)grid.x * grid.y <= 2LL * sms;
    const auto finish = wide ? (early ? few_rows_finish_kernel<T, true, true> : few_rows_finish_kernel<T, true, false>)
                             : (early ? few_rows_finish_kernel<T, false, true> : few_rows_finish_kernel<T, false, false>);
    const cudaError_t e = sgh::launch_early(finish, grid, 256, 0, c.stream, w, B, ad, bias, c.N % 4 == 0, c.H, (long long)c.ldh,
                                            static_cast<T *>(c.Y), (long long)c.ldy);
    if (e != cudaSuccess) return sgh::cuda_fail(e);
    if ((st = launched()) != SGEMM_OK) return st;
    return ws.release();
}

// Few rows: the rank side row by row (M rank (K + N) elements of the stack from L2, and
// partial sums of all of Y) against grouping it by adapter (four launches more, about 20
// us).  Both types cross over at the same rows, within what the rule gives away.  us, row by row /
// grouped, 8 adapters at random, bfloat16 and float32: 4096 x 4096 of rank 16, 128 rows 27 / 44 and
// 79 / 98, 256 rows 36 / 48 and 92 / 104, 512 rows 68 / 50 and 146 / 142; 1024 x 1024 of rank 64,
// 512 rows 26 / 40 and 42 / 50, 768 rows 37 / 44 and 53 / 55, 1000 rows 45 / 44 and 63 / 58; 768 x
// 768 of rank 16, 1280 rows 30 / 32 and 39 / 46; 512 x 512, 1280 rows 19 / 30 and 29 / 38.
bool few_rows(const Call &c) {
    if (c.K == 0 || c.N == 0) return false;
    if (c.M <= STREAM_ROWS) return true;
    if (c.L == 0) return c.M <= 256;
    const long long stack = (long long)c.M * c.R * ((long long)c.K + c.N);
    return c.M <= FEW_ROWS && stack <= 68000000 && (long long)c.M * c.N <= 1500000;
}

template <class T>
int forward(const Call &c) {
    int sms, st;
    cudaMemPool_t pool;
    if ((st = sgh::current_device(&sms, &pool)) != SGEMM_OK) return st;
    return few_rows(c) ? forward_few_rows<T>(c, sms, pool) : many_rows<T, false>(c, sms, pool);
}

template <class T>
int backward(const Call &c) {
    int sms, st;
    cudaMemPool_t pool;
    if ((st = sgh::current_device(&sms, &pool)) != SGEMM_OK) return st;
    return many_rows<T, true>(c, sms, pool);
}

template <class T>
int weight_grad(int M, int N, int K, Act8Rows x, const void *dY, int lddy, float beta, void *dW,
                int lddw, cudaStream_t stream) {
    int sms, st;
    cudaMemPool_t pool;
    if ((st = sgh::current_device(&sms, &pool)) != SGEMM_OK) return st;
    const sgp::Epilogue<T, false> epi{Adapters{}, nullptr, 0, {}, nullptr, beta, static_cast<T *>(dW), lddw};
    if (M == 0) return sgp::finish<T, false>(K, N, 0, nullptr, nullptr, epi, stream);
    Packed<T> D(M, N, dY, lddy);
    const sgp::Split split = sgp::plan_split(K, N, M, sizeof(T) == 4 ? 3 : 1, sms);
    const long long xpitch = pitch8(K);
    const size_t x_elems = size_t(M) * xpitch;
    sgh::Workspace ws(pool, stream);
    st = ws.allocate(sgh::Workspace::piece(x_elems * 2) + D.bytes() +
                     sgh::Workspace::piece(split.partial_floats * 4));
    if (st != SGEMM_OK) return st;
    const Parts xp{ws.take<bf16>(x_elems), xpitch, M * xpitch};
    D.place(ws);
    float *partial = split.partial_floats ? ws.take<float>(split.partial_floats) : nullptr;
    const PartsJob<Act8Rows> xjob(x, M, K, aligned(x.q, 8) && x.ldq % 8 == 0, xp);
    st = prepare<1, Packed<T>::PARTS>(M, Adapters{}, Groups{}, xjob, D.job(), sms, stream);
    if (st != SGEMM_OK) return st;
    sgp::Product g;
    g.M = K, g.N = N, g.K = M;
    g.a = {xp.p, K, M, 1, xpitch, M * xpitch};
    g.b = D.operand();
    if ((st = sgp::run<T, sgp::WEIGHT_GRAD>(g, epi, split, partial, sms, stream)) != SGEMM_OK) return st;
    return ws.release();
}

}  // namespace

cudaError_t sgh::lora_error_word(unsigned *v, bool clear) { return sgv::unit_error_word(v, clear); }

SGEMM_API int sgemm_lora(int type, int M, int N, int K, int L, int R, const void *X, int ldx,
                         const void *W, int ldw, const void *A, int lda, long long stride_a,
                         const void *B, int ldb, long long stride_b, const int *ids,
                         const int *ranks, const float *scales, const void *bias, float *H, int ldh,
                         void *Y, int ldy, sgemm_stream_t stream) {
    Call c{};
    c.type = type, c.M = M, c.N = N, c.K = K, c.L = L, c.R = R;
    c.X = X, c.ldx = ldx, c.W = W, c.ldw = ldw;
    c.A = A, c.lda = lda, c.stride_a = stride_a, c.B = B, c.ldb = ldb, c.stride_b = stride_b;
    c.ids = ids, c.ranks = ranks, c.scales = scales, c.bias = bias;
    c.H = H, c.ldh = ldh, c.Y = Y, c.ldy = ldy;
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    const int st = check_common(c);
    if (st != SGEMM_OK) return st;
    if (M == 0 || (N == 0 && !H)) return SGEMM_OK;
    const size_t size = element_bytes(type);
    if ((K > 0 && bad_matrix(X, ldx, K, size)) ||
        (K > 0 && N > 0 && bad_matrix(W, ldw, N, size)) || (N > 0 && bad_matrix(Y, ldy, N, size)) ||
        !aligned(bias, size))
        return SGEMM_ERR_INVALID_ARG;
    if (L > 0 && (bad_stack(A, lda, stride_a, L, K, R, size) ||
                  bad_stack(B, ldb, stride_b, L, R, N, size)))
        return SGEMM_ERR_INVALID_ARG;
    if (H && R > 0 && bad_matrix(H, ldh, R, 4)) return SGEMM_ERR_INVALID_ARG;
    if (L == 0 && H) {   // no row has an adapter
        const cudaError_t e = R <= 0 ? cudaSuccess
                                     : cudaMemset2DAsync(H, size_t(ldh) * 4, 0, size_t(R) * 4, size_t(M), c.stream);
        if (e != cudaSuccess) return sgh::cuda_fail(e);
        c.H = nullptr;
        if (N == 0) return SGEMM_OK;
    }
    return type == SGEMM_BF16 ? forward<bf16>(c) : forward<float>(c);
}

SGEMM_API int sgemm_lora_backward(int type, int M, int N, int K, int L, int R, const void *dY,
                                  int lddy, const void *X, int ldx, const signed char *q, int ldq,
                                  const signed char *e, int lde, const void *W, int ldw,
                                  const void *A, int lda, long long stride_a, const void *B, int ldb,
                                  long long stride_b, const int *ids, const int *ranks,
                                  const float *scales, const float *H, int ldh, void *dX, int lddx,
                                  void *dA, int ldda, long long stride_da, void *dB, int lddb,
                                  long long stride_db, sgemm_stream_t stream) {
    Call c{};
    c.type = type, c.M = M, c.N = N, c.K = K, c.L = L, c.R = R;
    c.dY = dY, c.lddy = lddy, c.X = X, c.ldx = ldx;
    c.q = q, c.ldq = ldq, c.e = e, c.lde = lde;
    c.W = W, c.ldw = ldw;
    c.A = A, c.lda = lda, c.stride_a = stride_a, c.B = B, c.ldb = ldb, c.stride_b = stride_b;
    c.ids = ids, c.ranks = ranks, c.scales = scales;
    c.H = const_cast<float *>(H), c.ldh = ldh;
    c.dX = dX, c.lddx = lddx;
    c.dA = dA, c.ldda = ldda, c.stride_da = stride_da;
    c.dB = dB, c.lddb = lddb, c.stride_db = stride_db;
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    const int st = check_common(c);
    if (st != SGEMM_OK) return st;
    if (L > 0 && K > 0 && N > 0 && (!dA) != (!dB)) return SGEMM_ERR_INVALID_ARG;
    const size_t size = element_bytes(type);
    const bool want_dx = dX && M > 0 && K > 0, want_stack = (dA || dB) && L > 0;
    if (M > 0 && N > 0 && (want_dx || want_stack) && bad_matrix(dY, lddy, N, size))
        return SGEMM_ERR_INVALID_ARG;
    if (want_dx && (bad_matrix(dX, lddx, K, size) || (N > 0 && bad_matrix(W, ldw, N, size))))
        return SGEMM_ERR_INVALID_ARG;
    if (L > 0 && (want_dx || want_stack) &&
        (bad_stack(A, lda, stride_a, L, K, R, size) || bad_stack(B, ldb, stride_b, L, R, N, size)))
        return SGEMM_ERR_INVALID_ARG;
    if (want_stack) {
        if (bad_stack(dA, ldda, stride_da, L, K, R, size) || bad_stack(dB, lddb, stride_db, L, R, N, size) ||
            (M > 0 && bad_matrix(H, ldh, R, 4)))
            return SGEMM_ERR_INVALID_ARG;
        if (M > 0 && K > 0 &&
            (X ? bad_matrix(X, ldx, K, size)
               : bad_matrix(q, ldq, K, 1) || bad_matrix(e, lde, blocks_of(K), 1)))
            return SGEMM_ERR_INVALID_ARG;
    }
    if (!want_dx && !want_stack) return SGEMM_OK;
    return type == SGEMM_BF16 ? backward<bf16>(c) : backward<float>(c);
}

SGEMM_API int sgemm_act8_weight_grad(int type, int M, int N, int K, const signed char *q, int ldq,
                                     const signed char *e, int lde, const void *dY, int lddy,
                                     float beta, void *dW, int lddw, sgemm_stream_t stream) {
    const int st = check_sizes(type, M, N, K);
    if (st != SGEMM_OK) return st;
    if (N == 0 || K == 0) return SGEMM_OK;
    const size_t size = element_bytes(type);
    if (bad_matrix(dW, lddw, N, size) ||
        (M > 0 && (bad_matrix(dY, lddy, N, size) || bad_matrix(q, ldq, K, 1) ||
                   bad_matrix(e, lde, blocks_of(K), 1))))
        return SGEMM_ERR_INVALID_ARG;
    const Act8Rows x{q, e, ldq, lde};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return type == SGEMM_BF16 ? weight_grad<bf16>(M, N, K, x, dY, lddy, beta, dW, lddw, s)
                              : weight_grad<float>(M, N, K, x, dY, lddy, beta, dW, lddw, s);
}
