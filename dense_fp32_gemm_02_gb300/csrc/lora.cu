// lora.cu -- entry points of the adapter layer and of the weight gradient from an
// 8-bit checkpoint: argument checks, workspaces and launches.
#include <algorithm>

#include "../../include/sgemm_layers.h"
#include "host_state.h"
#include "lora.cuh"
#include "parts_gemm.h"
#include "variant.cuh"

#define SGEMM_API extern "C" __attribute__((visibility("default")))

namespace {

using namespace sgl;

constexpr int kMaxRank = 128, kMaxAdapters = 1024;

bool aligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
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
long long pitch8(long long cols) { return (cols + 7) / 8 * 8; }

// A matrix that the TMA reads where it lies: bfloat16, 16-byte aligned rows.
template <class T>
bool in_place(const T *p, int ld) {
    return sizeof(T) == 2 && aligned(p, 16) && ld % 8 == 0;
}

// The parts of a rows x cols matrix as an operand: the matrix itself, or planes in the
// workspace that pack() fills.
template <class T>
struct Packed {
    static constexpr int PARTS = sizeof(T) == 4 ? 3 : 1;
    long long rows, cols, pitch;
    bool direct;
    const T *src;
    int ld;
    Parts parts{};

    Packed(long long rows_, long long cols_, const void *p, int ld_)
        : rows(rows_), cols(cols_), pitch(pitch8(cols_)), direct(in_place(static_cast<const T *>(p), ld_)),
          src(static_cast<const T *>(p)), ld(ld_) {}

    size_t elements() const { return direct ? 0 : size_t(PARTS) * rows * pitch; }
    size_t bytes() const { return sgh::Workspace::piece(elements() * 2); }
    void place(sgh::Workspace &ws) {
        if (!direct) parts = Parts{ws.take<bf16>(elements()), pitch, rows * pitch};
    }
    int pack(int sms, cudaStream_t stream) const {
        if (direct) return SGEMM_OK;
        const bool wide = aligned(src, 16) && ld % (16 / sizeof(T)) == 0;
        const long long threads = rows * (pitch / 8);
        const unsigned grid = unsigned(std::min<long long>((threads + 255) / 256, sms * 16LL));
        parts_kernel<PARTS><<<grid, 256, 0, stream>>>(int(rows), int(cols), Rows<T>{src, ld}, wide, parts);
        return launched();
    }
    sgp::Operand operand() const {
        if (direct)
            return {reinterpret_cast<const bf16 *>(src), cols, rows, 1, ld, rows * (long long)ld};
        return {parts.p, cols, rows, PARTS, pitch, rows * pitch};
    }
};

template <class T>
Stack<const T> stack_of(const void *p, int ld, long long stride) {
    return {static_cast<const T *>(p), ld, stride};
}

// out (M x N) = P * Q + rank-side term of X's (forward) or dY's (backward) rows.
//   forward:  P = X (M x K), Q = W (K x N), S = scale X A, V = B
//   backward: P = dY, Q = W^T (N x K stored), S = G, V = A^T
// `S`, where given, receives the rank-side sums for the caller.
template <class T, bool BACK>
int projection(const Call &c, float *S, float *H, int ldh, void *out, int ldo, bool want_out) {
    int sms, st;
    cudaMemPool_t pool;
    if ((st = sgh::current_device(&sms, &pool)) != SGEMM_OK) return st;
    const Adapters ad = c.adapters();
    const int M = c.M, N = BACK ? c.K : c.N, K = BACK ? c.N : c.K;
    const bool ranked = c.L > 0, product = want_out && K > 0 && N > 0;
    constexpr auto LAYOUT = BACK ? sgp::INPUT_GRAD : sgp::FORWARD;
    constexpr int PRODUCTS = sizeof(T) == 4 ? 6 : 1, S_PARTS = sizeof(T) == 4 ? 3 : 2;
    Packed<T> P(M, K, BACK ? c.dY : c.X, BACK ? c.lddy : c.ldx), Q(c.K, c.N, c.W, c.ldw);
    const sgp::Split split = product ? sgp::plan_split(M, N, K, PRODUCTS, sms) : sgp::Split{0, 0};
    const bool slabs = ranked && product && split.splits == 1;   // the rank side in the MMA loop
    const int tiles = (M + 255) / 256, slots = std::min(c.L, tiles);
    const long long rpitch = pitch8(c.R);
    const long long vrows = BACK ? N : c.R, vcols = BACK ? c.R : N, vpitch = pitch8(vcols);

    sgh::Workspace ws(pool, c.stream);
    const auto piece = [](size_t n) { return sgh::Workspace::piece(n); };
    const size_t s_floats = ranked && !S ? size_t(M) * c.R : 0;
    const size_t h_elems = slabs ? size_t(S_PARTS) * M * rpitch : 0;
    const size_t v_elems = slabs ? size_t(Packed<T>::PARTS) * slots * vrows * vpitch : 0;
    st = ws.allocate(piece(s_floats * 4) + piece(h_elems * 2) + piece(v_elems * 2) +
                     (slabs ? piece(tiles * 4) + piece(slots * 4) : 0) +
                     (product ? P.bytes() + Q.bytes() + piece(split.partial_floats * 4) : 0));
    if (st != SGEMM_OK) return st;
    RankSide side{S, c.R, H, ldh, Parts{}};
    if (s_floats) side.S = ws.take<float>(s_floats);
    int *tile_adapter = nullptr, *slot_adapter = nullptr;
    Parts v{};
    if (slabs) {
        side.parts = Parts{ws.take<bf16>(h_elems), rpitch, M * rpitch};
        v = Parts{ws.take<bf16>(v_elems), vpitch, vrows * vpitch};
        tile_adapter = ws.take<int>(tiles);
        slot_adapter = ws.take<int>(slots);
    }
    const Stack<const T> A = stack_of<T>(c.A, c.lda, c.stride_a), B = stack_of<T>(c.B, c.ldb, c.stride_b);
    if (ranked) {
        const long long pairs = (long long)M * c.R;
        const Rows<T> X{P.src, P.ld};
        rank_side_kernel<T, BACK><<<unsigned((pairs + 7) / 8), 256, 0, c.stream>>>(M, K, X, BACK ? B : A, ad, side);
        if ((st = launched()) != SGEMM_OK) return st;
    }
    if (!want_out || N == 0) return ws.release();
    sgp::Epilogue<T, BACK> epi{ad, side.S, side.lds, BACK ? A : B, BACK ? nullptr : static_cast<const T *>(c.bias),
                               0.0f, static_cast<T *>(out), ldo};
    if (!product) {   // K == 0: the epilogue of a zero sum
        if ((st = sgp::finish<T, BACK>(M, N, 0, nullptr, epi, c.stream)) != SGEMM_OK) return st;
        return ws.release();
    }
    if (slabs) {
        tile_adapters_kernel<<<1, 1024, 0, c.stream>>>(M, tiles, slots, ad, tile_adapter, slot_adapter);
        if ((st = launched()) != SGEMM_OK) return st;
        const long long threads = vrows * (vpitch / 8);
        const dim3 grid(unsigned(std::min<long long>((threads + 255) / 256, sms * 4LL)), unsigned(slots));
        pack_stack_kernel<T, !BACK><<<grid, 256, 0, c.stream>>>(int(vrows), int(vcols), BACK ? A : B, ad,
                                                               slot_adapter, slots, v);
        if ((st = launched()) != SGEMM_OK) return st;
    }
    P.place(ws);
    Q.place(ws);
    float *partial = split.partial_floats ? ws.take<float>(split.partial_floats) : nullptr;
    if ((st = P.pack(sms, c.stream)) != SGEMM_OK || (st = Q.pack(sms, c.stream)) != SGEMM_OK) return st;
    sgp::Product g;
    g.M = M, g.N = N, g.K = K;
    g.a = P.operand();
    g.b = Q.operand();
    if (slabs) {
        g.h = {side.parts.p, c.R, M, S_PARTS, rpitch, M * rpitch};
        g.v = {v.p, vcols, vrows, (long long)Packed<T>::PARTS * slots, vpitch, vrows * vpitch};
        g.slots = slots;
        g.tile_adapter = tile_adapter;
    }
    if ((st = sgp::run<T, LAYOUT>(g, epi, split, partial, sms, c.stream)) != SGEMM_OK) return st;
    return ws.release();
}

template <class T>
int forward(const Call &c) {
    return projection<T, false>(c, nullptr, c.H, c.ldh, c.Y, c.ldy, true);
}

template <class T>
int backward(const Call &c) {
    int sms, st;
    cudaMemPool_t pool;
    if ((st = sgh::current_device(&sms, &pool)) != SGEMM_OK) return st;
    const Adapters ad = c.adapters();
    const bool want_dx = c.dX && c.M > 0 && c.K > 0, want_stack = (c.dA || c.dB) && c.L > 0;
    sgh::Workspace ws(pool, c.stream);
    float *G = nullptr;
    if (c.L > 0 && c.M > 0) {
        if ((st = ws.allocate(sgh::Workspace::piece(size_t(c.M) * c.R * 4))) != SGEMM_OK) return st;
        G = ws.take<float>(size_t(c.M) * c.R);
    }
    if (c.M > 0 && (st = projection<T, true>(c, G, nullptr, 0, c.dX, c.lddx, want_dx)) != SGEMM_OK) return st;
    if (want_stack) {
        if (c.K > 0) {
            const dim3 grid(unsigned((c.K + 255) / 256), unsigned(c.R), unsigned(c.L));
            const Stack<T> out{static_cast<T *>(c.dA), c.ldda, c.stride_da};
            if (c.X)
                stack_grad_kernel<T, false><<<grid, 256, 0, c.stream>>>(
                    c.M, c.K, Rows<T>{static_cast<const T *>(c.X), c.ldx}, G, c.R, ad, false, out);
            else
                stack_grad_kernel<T, false><<<grid, 256, 0, c.stream>>>(
                    c.M, c.K, Act8Rows{c.q, c.e, c.ldq, c.lde}, G, c.R, ad, false, out);
            if ((st = launched("lora backward")) != SGEMM_OK) return st;
        }
        if (c.N > 0) {
            const dim3 grid(unsigned((c.N + 255) / 256), unsigned(c.R), unsigned(c.L));
            stack_grad_kernel<T, true><<<grid, 256, 0, c.stream>>>(
                c.M, c.N, Rows<T>{static_cast<const T *>(c.dY), c.lddy}, c.H, c.ldh, ad, true,
                Stack<T>{static_cast<T *>(c.dB), c.lddb, c.stride_db});
            if ((st = launched("lora backward")) != SGEMM_OK) return st;
        }
    }
    return ws.release();
}

template <class T>
int weight_grad(int M, int N, int K, Act8Rows x, const void *dY, int lddy, float beta, void *dW,
                int lddw, cudaStream_t stream) {
    int sms, st;
    cudaMemPool_t pool;
    if ((st = sgh::current_device(&sms, &pool)) != SGEMM_OK) return st;
    const sgp::Epilogue<T, false> epi{Adapters{}, nullptr, 0, {}, nullptr, beta, static_cast<T *>(dW), lddw};
    if (M == 0) return sgp::finish<T, false>(K, N, 0, nullptr, epi, stream);
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
    const bool wide = aligned(x.q, 8) && x.ldq % 8 == 0;
    const unsigned grid = unsigned(std::min<long long>((M * (xpitch / 8) + 255) / 256, sms * 16LL));
    parts_kernel<1><<<grid, 256, 0, stream>>>(M, K, x, wide, xp);
    if ((st = launched()) != SGEMM_OK || (st = D.pack(sms, stream)) != SGEMM_OK) return st;
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
    if (M == 0 || (N == 0 && (!H || L == 0))) return SGEMM_OK;
    const size_t size = element_bytes(type);
    if ((K > 0 && bad_matrix(X, ldx, K, size)) ||
        (K > 0 && N > 0 && bad_matrix(W, ldw, N, size)) || (N > 0 && bad_matrix(Y, ldy, N, size)) ||
        !aligned(bias, size))
        return SGEMM_ERR_INVALID_ARG;
    if (L > 0 && (bad_stack(A, lda, stride_a, L, K, R, size) ||
                  bad_stack(B, ldb, stride_b, L, R, N, size) || (H && bad_matrix(H, ldh, R, 4))))
        return SGEMM_ERR_INVALID_ARG;
    if (L == 0) c.H = nullptr;
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
