// norm.cu -- entry points of the root-mean-square norm, forward and backward, and rows in 8 bits
// for the product that reads them.
#include "layer_host.h"
#include "norm.cuh"
#include "variant.cuh"

#define SGEMM_API extern "C" __attribute__((visibility("default")))

namespace {

using namespace sgl;

template <class C>
using Kernel = void (*)(const C);

// A group of threads to a row, and how many rows to a block of so many threads.
template <class C>
struct Form {
    Kernel<C> kernel;
    int threads, rows;
    size_t smem = 0;
};

template <class T, int KIND, int THREADS, int CHUNKS, bool WIDE, bool LONG = false>
Form<NormCall<T>> form() {
    return {&norm_kernel<T, KIND, THREADS, CHUNKS, WIDE, LONG>, norm_block(THREADS), norm_block(THREADS) / THREADS};
}
// us, a warp to a row / four warps: y from 8192 x 1024 bfloat16 7.4 / 9.1, in 8 bits with residual 14.7 /
// 17.6; float32 12.1 / 11.4 and 22.0 / 20.1; 4097 x 1023 (one element at a time) 8.7 / 7.8 and 21.5 / 12.9.
// 8192 x 2048 bfloat16 in 8 bits with residual, 256 threads of two pieces / one 44.5 / 34.9; of 4096 columns two pieces
// 51.5, 512 threads of one 78.8.
template <class T, int KIND, bool WIDE>
Form<NormCall<T>> forward_form(int M, int K, int sms) {
    if (K <= 256) return form<T, KIND, 32, 1, WIDE>();
    if (WIDE && M <= sms && K <= 8192)   // a block to an SM: as many threads as there is work for
        return K <= 2048 ? form<T, KIND, 256, 1, true>() : form<T, KIND, 1024, 1, true>();
    if (K <= 1024) {
        if constexpr (WIDE && sizeof(T) == 2) return form<T, KIND, 32, 4, true>();
        else return form<T, KIND, 128, 1, WIDE>();
    }
    if (K <= 2048) return form<T, KIND, 256, 1, WIDE>();
    if (K <= 4096) return form<T, KIND, 256, 2, WIDE>();
    if (WIDE && K <= 8192) return form<T, KIND, 256, 4, true>();
    if (K <= 16384) return form<T, KIND, 512, 4, WIDE>();
    return form<T, KIND, 512, 4, WIDE, true>();
}

template <class T, int KIND>
int forward(const NormCall<T> &c, int sms, cudaStream_t stream) {
    const bool wide = c.K % 8 == 0 && sgh::wide_rows(c.X, c.ldx) && sgh::wide_rows(c.R, c.ldr) &&
                      sgh::wide_rows(c.S, c.lds) && sgh::wide_rows(c.Y, c.ldy) && sgh::aligned(c.w, 16) &&
                      sgh::aligned(c.q, 8) && c.ldq % 8 == 0;
    const auto f = wide ? forward_form<T, KIND, true>(c.M, c.K, sms) : forward_form<T, KIND, false>(c.M, c.K, sms);
    return sgh::launch(wide ? "norm, rows read 16 bytes at a time" : "norm, any alignment", f.kernel,
                       dim3(unsigned((c.M + f.rows - 1LL) / f.rows)), unsigned(f.threads), 0, stream, c);
}

template <class T, int THREADS, int CHUNKS, bool WIDE, bool LONG = false>
Form<NormBackCall<T>> back_form() {
    return {&norm_backward_kernel<T, THREADS, CHUNKS, WIDE, LONG>, norm_block(THREADS), norm_block(THREADS) / THREADS,
            NormRing<T, THREADS, CHUNKS, WIDE, LONG>::BYTES};
}
template <class T, bool WIDE>
Form<NormBackCall<T>> backward_form(int K) {
    return K <= 256     ? back_form<T, 32, 1, WIDE>()
           : K <= 1024  ? back_form<T, 128, 1, WIDE>()
           : K <= 4096  ? back_form<T, 256, 2, WIDE>()
           : K <= 8192  ? back_form<T, 512, 2, WIDE>()
           : K <= 16384 ? back_form<T, 512, 4, WIDE>()
                        : back_form<T, 512, 4, WIDE, true>();
}

template <class T>
int backward(NormBackCall<T> c, T *dw, cudaStream_t stream) {
    int sms, st;
    cudaMemPool_t pool;
    if ((st = sgh::current_device(&sms, &pool)) != SGEMM_OK) return st;
    if (c.M == 0) {   // no row: dw is zero
        const cudaError_t e = dw ? cudaMemsetAsync(dw, 0, size_t(c.K) * sizeof(T), stream) : cudaSuccess;
        return e == cudaSuccess ? SGEMM_OK : sgh::cuda_fail(e);
    }
    const bool wide = c.K % 8 == 0 && sgh::wide_rows(c.dY, c.lddy) && sgh::wide_rows(c.V, c.ldv) &&
                      sgh::wide_rows(c.dS, c.ldds) && sgh::wide_rows(c.dX, c.lddx) && sgh::aligned(c.w, 16);
    const auto f = wide ? backward_form<T, true>(c.K) : backward_form<T, false>(c.K);
    int per_sm = 1;
    cudaError_t e = cudaFuncSetAttribute(f.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(f.smem));
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, f.kernel, f.threads, f.smem);
    if (e != cudaSuccess) return sgh::cuda_fail(e);
    const int blocks = int(std::min<long long>((c.M + f.rows - 1LL) / f.rows, (long long)sms * std::max(1, per_sm)));
    sgh::Workspace ws(pool, stream);
    const size_t floats = dw ? size_t(blocks) * c.K : 0;
    if ((st = ws.allocate(sgh::Workspace::piece(floats * 4))) != SGEMM_OK) return st;
    c.partial = dw ? ws.take<float>(floats) : nullptr;
    st = sgh::launch(wide ? "norm backward, rows read 16 bytes at a time" : "norm backward, any alignment", f.kernel,
                     dim3(unsigned(blocks)), unsigned(f.threads), f.smem, stream, c);
    if (st != SGEMM_OK) return st;
    if (dw) {
        st = sgh::launch(nullptr, norm_weight_kernel<T>, dim3(unsigned((c.K + 31LL) / 32)), 1024, 0, stream, c.K, blocks,
                         (const float *)c.partial, dw);
        if (st != SGEMM_OK) return st;
    }
    return ws.release();
}

template <class T>
int forward_typed(NormCall<T> c, cudaStream_t stream) {
    int sms, st;
    cudaMemPool_t pool;
    if ((st = sgh::current_device(&sms, &pool)) != SGEMM_OK) return st;
    return c.q ? forward<T, NORM8>(c, sms, stream) : forward<T, NORM>(c, sms, stream);
}

template <class T>
NormCall<T> call_of(int M, int K, const void *X, int ldx, const void *R, int ldr, const void *w, float eps, void *S,
                    int lds, void *Y, int ldy, signed char *q, long long ldq, float *scale) {
    NormCall<T> c{};
    c.M = M, c.K = K, c.eps = eps;
    c.X = static_cast<const T *>(X), c.R = static_cast<const T *>(R), c.w = static_cast<const T *>(w);
    c.S = static_cast<T *>(S), c.Y = static_cast<T *>(Y);
    c.q = q, c.scale = scale;
    c.ldx = ldx, c.ldr = ldr, c.lds = lds, c.ldy = ldy, c.ldq = ldq;
    return c;
}

template <class T>
NormBackCall<T> back_call_of(int M, int K, const void *dY, int lddy, const void *V, int ldv, const void *w, float eps,
                             const void *dS, int ldds, void *dX, int lddx) {
    NormBackCall<T> c{};
    c.M = M, c.K = K, c.eps = eps;
    c.dY = static_cast<const T *>(dY), c.V = static_cast<const T *>(V), c.w = static_cast<const T *>(w);
    c.dS = static_cast<const T *>(dS), c.dX = static_cast<T *>(dX);
    c.lddy = lddy, c.ldv = ldv, c.ldds = ldds, c.lddx = lddx;
    return c;
}

// Rows of no columns: their scales alone are to be written, zeros.
int no_columns(int M, float *scale, cudaStream_t stream) {
    if (!scale) return SGEMM_OK;
    if (!sgh::aligned(scale, 4)) return SGEMM_ERR_INVALID_ARG;
    int sms, st;
    cudaMemPool_t pool;
    if ((st = sgh::current_device(&sms, &pool)) != SGEMM_OK) return st;
    const cudaError_t e = cudaMemsetAsync(scale, 0, size_t(M) * sizeof(float), stream);
    return e == cudaSuccess ? SGEMM_OK : sgh::cuda_fail(e);
}

}  // namespace

cudaError_t sgh::norm_error_word(unsigned *v, bool clear) { return sgv::unit_error_word(v, clear); }

int sgh::rows8(int type, int M, int K, const void *X, int ldx, signed char *q, long long ldq, float *scale, int sms,
               cudaStream_t stream) {
    const auto all = [&](auto c) { return forward<std::remove_const_t<std::remove_pointer_t<decltype(c.X)>>, ROWS8>(c, sms, stream); };
    return type == SGEMM_BF16
               ? all(call_of<bf16>(M, K, X, ldx, nullptr, 0, nullptr, 0.0f, nullptr, 0, nullptr, 0, q, ldq, scale))
               : all(call_of<float>(M, K, X, ldx, nullptr, 0, nullptr, 0.0f, nullptr, 0, nullptr, 0, q, ldq, scale));
}

SGEMM_API int sgemm_rmsnorm(int type, int M, int K, const void *X, int ldx, const void *R, int ldr, const void *w,
                            float eps, void *S, int lds, void *Y, int ldy, signed char *q, int ldq, float *scale,
                            sgemm_stream_t stream) {
    const int st = sgh::check_sizes(type, {M, K});
    if (st != SGEMM_OK) return st;
    if (!(eps >= 0.0f && eps <= 3.0e38f)) return SGEMM_ERR_INVALID_ARG;
    if (M == 0) return SGEMM_OK;
    if (K == 0) return no_columns(M, scale, reinterpret_cast<cudaStream_t>(stream));
    if ((!S && !Y && !q) || !q != !scale) return SGEMM_ERR_INVALID_ARG;
    const size_t size = sgh::element_bytes(type);
    if (sgh::bad_matrix(X, ldx, K, size) || sgh::bad_vector(w, size) || sgh::bad_optional(R, ldr, K, size) ||
        sgh::bad_optional(S, lds, K, size) || sgh::bad_optional(Y, ldy, K, size) || sgh::bad_optional(q, ldq, K, 1) ||
        !sgh::aligned(scale, 4) || (S && S == Y))
        return SGEMM_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return type == SGEMM_BF16
               ? forward_typed(call_of<bf16>(M, K, X, ldx, R, ldr, w, eps, S, lds, Y, ldy, q, ldq, scale), s)
               : forward_typed(call_of<float>(M, K, X, ldx, R, ldr, w, eps, S, lds, Y, ldy, q, ldq, scale), s);
}

SGEMM_API int sgemm_rmsnorm_backward(int type, int M, int K, const void *dY, int lddy, const void *V, int ldv,
                                     const void *w, float eps, const void *dS, int ldds, void *dX, int lddx, void *dw,
                                     sgemm_stream_t stream) {
    const int st = sgh::check_sizes(type, {M, K});
    if (st != SGEMM_OK) return st;
    if (!(eps >= 0.0f && eps <= 3.0e38f)) return SGEMM_ERR_INVALID_ARG;
    if (K == 0) return SGEMM_OK;
    const size_t size = sgh::element_bytes(type);
    if (!sgh::aligned(dw, size)) return SGEMM_ERR_INVALID_ARG;
    if (M > 0 && (sgh::bad_matrix(dY, lddy, K, size) || sgh::bad_matrix(V, ldv, K, size) || sgh::bad_vector(w, size) ||
                  sgh::bad_optional(dS, ldds, K, size) || sgh::bad_matrix(dX, lddx, K, size)))
        return SGEMM_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return type == SGEMM_BF16
               ? backward(back_call_of<bf16>(M, K, dY, lddy, V, ldv, w, eps, dS, ldds, dX, lddx), static_cast<bf16 *>(dw), s)
               : backward(back_call_of<float>(M, K, dY, lddy, V, ldv, w, eps, dS, ldds, dX, lddx), static_cast<float *>(dw), s);
}
