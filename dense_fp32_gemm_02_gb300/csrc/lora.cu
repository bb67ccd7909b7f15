// lora.cu -- entry points of the adapter layer and of the weight gradient from an
// 8-bit checkpoint: argument checks, workspaces and launches.
#include <algorithm>

#include "../../include/sgemm_layers.h"
#include "host_state.h"
#include "lora.cuh"

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

template <class T>
int forward(const Call &c) {
    int sms, st;
    cudaMemPool_t pool;
    if ((st = sgh::current_device(&sms, &pool)) != SGEMM_OK) return st;
    const Adapters ad = c.adapters();
    const Rows<T> X{static_cast<const T *>(c.X), c.ldx};
    const Stack<const T> A{static_cast<const T *>(c.A), c.lda, c.stride_a};
    const Stack<const T> B{static_cast<const T *>(c.B), c.ldb, c.stride_b};
    sgh::Workspace ws(pool, c.stream);
    float *S = c.H;
    long long lds = c.ldh;
    if (!S && c.L > 0) {
        if ((st = ws.allocate(sgh::Workspace::piece(size_t(c.M) * c.R * 4))) != SGEMM_OK) return st;
        S = ws.take<float>(size_t(c.M) * c.R);
        lds = c.R;
    }
    if (c.L > 0) {
        const long long pairs = (long long)c.M * c.R;
        rank_side_kernel<T, false><<<unsigned((pairs + 7) / 8), 256, 0, c.stream>>>(
            c.M, c.K, X, A, ad, false, S, lds);
        if ((st = launched()) != SGEMM_OK) return st;
    }
    if (c.N > 0) {
        const dim3 grid(unsigned((c.N + 63) / 64), unsigned((c.M + 63) / 64));
        const Expand<T, false> expand{ad, S, lds, B, true};
        product_kernel<<<grid, 256, 0, c.stream>>>(c.M, c.N, c.K, X,
                                                   Rows<T>{static_cast<const T *>(c.W), c.ldw},
                                                   expand, static_cast<const T *>(c.bias), 0.0f,
                                                   static_cast<T *>(c.Y), c.ldy);
        if ((st = launched("lora forward")) != SGEMM_OK) return st;
    }
    return ws.release();
}

template <class T>
int backward(const Call &c) {
    int sms, st;
    cudaMemPool_t pool;
    if ((st = sgh::current_device(&sms, &pool)) != SGEMM_OK) return st;
    const Adapters ad = c.adapters();
    const Rows<T> dY{static_cast<const T *>(c.dY), c.lddy};
    const Stack<const T> A{static_cast<const T *>(c.A), c.lda, c.stride_a};
    const Stack<const T> B{static_cast<const T *>(c.B), c.ldb, c.stride_b};
    sgh::Workspace ws(pool, c.stream);
    float *G = nullptr;
    if (c.L > 0 && c.M > 0) {
        if ((st = ws.allocate(sgh::Workspace::piece(size_t(c.M) * c.R * 4))) != SGEMM_OK) return st;
        G = ws.take<float>(size_t(c.M) * c.R);
        const long long pairs = (long long)c.M * c.R;
        rank_side_kernel<T, true><<<unsigned((pairs + 7) / 8), 256, 0, c.stream>>>(
            c.M, c.N, dY, B, ad, true, G, c.R);
        if ((st = launched()) != SGEMM_OK) return st;
    }
    if (c.dX && c.M > 0 && c.K > 0) {
        const dim3 grid(unsigned((c.K + 63) / 64), unsigned((c.M + 63) / 64));
        const Expand<T, true> expand{ad, G, c.R, A, false};
        product_kernel<<<grid, 256, 0, c.stream>>>(c.M, c.K, c.N, dY,
                                                   Transposed<T>{static_cast<const T *>(c.W), c.ldw},
                                                   expand, static_cast<const T *>(nullptr), 0.0f,
                                                   static_cast<T *>(c.dX), c.lddx);
        if ((st = launched("lora backward")) != SGEMM_OK) return st;
    }
    if ((c.dA || c.dB) && c.L > 0) {
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
                c.M, c.N, dY, c.H, c.ldh, ad, true,
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
    const dim3 grid(unsigned((N + 63) / 64), unsigned((K + 63) / 64));
    product_kernel<<<grid, 256, 0, stream>>>(K, N, M, Act8Transposed{x},
                                             Rows<T>{static_cast<const T *>(dY), lddy}, NoExpand{},
                                             static_cast<const T *>(nullptr), beta,
                                             static_cast<T *>(dW), lddw);
    return launched("act8 weight gradient");
}

}  // namespace

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
