/*
 * sgemm_layers.h -- the linear layer of a language model around the GEMM of
 * sgemm.h: low-rank adapters of many requests beside a shared projection
 * (forward and backward), activation checkpoints in 8 bits with their use
 * in the backward pass, the root-mean-square norm before such a layer, with an
 * output in 8 bits and the projection that reads it, and the gated feed-forward
 * block.  Part of libsgemm.so; statuses, streams, ownership,
 * workspaces and the device error word are those of sgemm.h.
 *
 * Conventions of every entry point here:
 *  - `type` is the element type of the activations, weights and gradients
 *    (sgemm_type); all of a call's matrices have it unless a parameter says
 *    otherwise.  Sums are fp32 and each output is rounded once.  (The tensor
 *    cores truncate where they add: bfloat16 sums of up to 8192 terms, which
 *    stays under 3e-5 of the terms' magnitudes, and float32 sums of up to 512;
 *    what is longer is added to nearest.)
 *  - Matrices are row-major with a leading dimension in elements, at least
 *    max(1, columns).  Pointers must be aligned to their element (16-byte
 *    aligned rows are faster, no more).
 *  - Sizes are at most 2^31 - 65536 (SGEMM_ERR_TOO_LARGE above that).
 *  - Elements of an output outside its rows x columns block are not written.
 *  - Infinities and NaNs give what the formulas give, however many rows there
 *    are.  float32 magnitudes below 2^-110 may count as the next lower multiple
 *    of 2^-133, and next to an infinity a value under 2^-96 as zero.
 *  - Results are bitwise reproducible from call to call on a GPU model.
 *  - The work is enqueued on `stream`; nothing synchronises the host.  Workspaces come
 *    from the library's stream-ordered pool and go back to it behind the last kernel.
 *    Every call may be captured in a graph after a first call on the device.
 */
#ifndef DENSE_FP32_GEMM_02_GB300_SGEMM_LAYERS_H
#define DENSE_FP32_GEMM_02_GB300_SGEMM_LAYERS_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SGEMM_F32 = 0,  /* IEEE binary32 */
    SGEMM_BF16 = 1  /* bfloat16 */
} sgemm_type;

/* ------------------------------------------------------------------ adapters
 *
 * A stack of L low-rank adapters of rank at most R beside one projection W
 * (K x N).  Row i of X (M x K) uses adapter a = ids[i]; a row whose id is not in
 * [0, L) uses none.
 *
 *   A: L matrices K x R, `stride_a` elements apart (row pitch lda >= R)
 *   B: L matrices R x N, `stride_b` elements apart (row pitch ldb >= N)
 *   ids: M ints on the device
 *   ranks: L ints on the device, or NULL (every rank is R).  Only the first
 *          min(max(ranks[a], 0), R) columns of A_a and rows of B_a are used:
 *          what the stack holds past them, NaN included, reaches no result.
 *   scales: L floats on the device, or NULL (1)
 *
 * An adapter's values reach the rows that use it and no others: a row without
 * an adapter is exactly the plain projection whatever the stack holds.
 * 1 <= R <= 128 where L > 0; 0 <= L <= 1024.  L == 0 is the plain projection.
 */

/*
 * sgemm_lora -- forward, for one token up to a long prefill:
 *
 *   H[i] = X[i] * A_a                                     (M x R, fp32)
 *   Y[i] = X[i] * W + bias + scales[a] * H[i] * B_a       (M x N)
 *
 * bias: N elements of `type`, or NULL.  H (row pitch ldh >= R), where it is not
 * NULL, receives X * A_a for the backward pass: zero in the columns past an
 * adapter's rank and in rows without one.  Y must not overlap an input.
 * M == 0 or N == 0 leaves Y alone (H is still written where M > 0, by zeros where
 * L == 0).
 */
int sgemm_lora(int type, int M, int N, int K, int L, int R,
               const void *X, int ldx,
               const void *W, int ldw,
               const void *A, int lda, long long stride_a,
               const void *B, int ldb, long long stride_b,
               const int *ids, const int *ranks, const float *scales,
               const void *bias,
               float *H, int ldh,
               void *Y, int ldy,
               sgemm_stream_t stream);

/*
 * sgemm_lora_backward -- the gradients of sgemm_lora for dY (M x N), W frozen:
 *
 *   G[i]  = scales[a] * dY[i] * B_a^T
 *   dX[i] = dY[i] * W^T + G[i] * A_a^T                    (M x K)
 *   dA_a  = sum over the rows i of a of X[i]^T * G[i]     (K x R each)
 *   dB_a  = sum over the rows i of a of scales[a] * H[i]^T * dY[i]   (R x N each)
 *
 * H is what the forward call wrote.  X is given as the matrix (X, ldx), or with
 * X == NULL as its 8-bit checkpoint (q, ldq, e, lde; see below).  dX may be
 * NULL, and dA may be NULL together with dB: those are not computed, and the
 * inputs that only they need (W and dX; X and H) are not read.  dA and dB are
 * written whole: zero past an adapter's rank and for adapters without rows.
 * The outputs must not overlap an input or each other.
 */
int sgemm_lora_backward(int type, int M, int N, int K, int L, int R,
                        const void *dY, int lddy,
                        const void *X, int ldx,
                        const signed char *q, int ldq, const signed char *e, int lde,
                        const void *W, int ldw,
                        const void *A, int lda, long long stride_a,
                        const void *B, int ldb, long long stride_b,
                        const int *ids, const int *ranks, const float *scales,
                        const float *H, int ldh,
                        void *dX, int lddx,
                        void *dA, int ldda, long long stride_da,
                        void *dB, int lddb, long long stride_db,
                        sgemm_stream_t stream);

/* ------------------------------------------------------------------ checkpoints
 *
 * The 8-bit form of a matrix (M x K): q, M x K int8, and e, M x ceil(K/32) int8,
 * one exponent for each block of 32 columns of a row (the last one of a row may
 * be shorter).  With t the largest magnitude of a block, e is the least integer
 * >= -126 with t <= 127 * 2^e and q = x / 2^e rounded to the nearest integer,
 * ties to even; the element stands for q * 2^e, which float32 and bfloat16 hold
 * exactly.  (Past 127 * 2^121, 0.8 % below the largest float32, e stays 121 and
 * q stops at 127 in magnitude.)  A block with an infinity or a NaN is kept as e = -128, q = 0 and
 * stands for NaN throughout.
 */

/*
 * sgemm_act8_store -- the checkpoint of Z, and with it Y = act(Z) (sgemm_act of
 * sgemm.h) in the same pass where Y is not NULL.  Y may be Z itself (same
 * pointer and leading dimension).  GELU is +inf at +inf and, 0 times infinity, NaN at
 * -inf, as its formula is; a NaN stays one under either activation (sgemm_ex's RELU
 * gives 0).
 */
int sgemm_act8_store(int type, int M, int K, const void *Z, int ldz, int act,
                     signed char *q, int ldq, signed char *e, int lde,
                     void *Y, int ldy, sgemm_stream_t stream);

/* sgemm_act8_load -- X = the values that a checkpoint stands for. */
int sgemm_act8_load(int type, int M, int K,
                    const signed char *q, int ldq, const signed char *e, int lde,
                    void *X, int ldx, sgemm_stream_t stream);

/*
 * sgemm_act8_grad -- dZ = dY * act'(z), z the values of a checkpoint (of the
 * activation's input).  relu'(0) is 0.  dZ is NaN where z is.  dZ may be dY
 * itself (same pointer and leading dimension).
 */
int sgemm_act8_grad(int type, int M, int K,
                    const signed char *q, int ldq, const signed char *e, int lde, int act,
                    const void *dY, int lddy, void *dZ, int lddz, sgemm_stream_t stream);

/*
 * sgemm_act8_weight_grad -- dW = x^T * dY + beta * dW (K x N), x (M x K) the
 * values of a checkpoint, dY M x N.  dW is not read when beta == 0.  M == 0
 * gives dW = beta * dW.
 */
int sgemm_act8_weight_grad(int type, int M, int N, int K,
                           const signed char *q, int ldq, const signed char *e, int lde,
                           const void *dY, int lddy, float beta, void *dW, int lddw,
                           sgemm_stream_t stream);

/* ------------------------------------------------------------------ norm and rows in 8 bits
 *
 * A matrix (M x K) in rows of 8 bits: q, M x K int8, and scale, M floats; row i stands for
 * scale[i] * q[i].  With t the largest magnitude of a row, scale = t / 127 and q = x / scale rounded to
 * the nearest integer, ties to even, of the exact quotient.  A row of zeros has scale 0, one of no
 * columns too; a row with an infinity or a NaN is kept as q = 0, scale NaN and stands for NaN
 * throughout.
 */

/*
 * sgemm_rmsnorm -- the root-mean-square norm of the rows of V = X + R, and V itself:
 *
 *   V = X + R (rounded to `type`: the residual stream as it is held; X where R is NULL)
 *   y[j] = V[j] * w[j] / sqrt(mean over the row of V^2 + eps)
 *
 * w: K elements of `type`.  Outputs, each of which may be NULL but not all: S receives V; Y receives y
 * in `type`; (q, scale), NULL together, receive y as rows of 8 bits (of the values before they are
 * rounded to `type`).  S and Y may be X or R (same pointer and leading dimension), not each other.
 * eps >= 0.  The mean is taken where squares leave fp32's range too; a row with an infinity has y = 0
 * where V is finite, and NaN at the infinity.
 */
int sgemm_rmsnorm(int type, int M, int K,
                  const void *X, int ldx,
                  const void *R, int ldr,
                  const void *w, float eps,
                  void *S, int lds,
                  void *Y, int ldy,
                  signed char *q, int ldq, float *scale,
                  sgemm_stream_t stream);

/*
 * sgemm_rmsnorm_backward -- the gradients of sgemm_rmsnorm's y for dY (M x K), given V:
 * with r = 1 / sqrt(mean(V^2) + eps), n = V r and g = dY w,
 *
 *   dX[j] = dS[j] + r * (g[j] - n[j] * mean over the row of g n)
 *   dw[j] = sum over the rows of dY[j] * n[j]
 *
 * dX is the gradient of X and of R alike.  dS, the gradient that reaches V by its other way (the
 * residual stream), may be NULL (0); dw (K elements) may be NULL.  M == 0 gives dw = 0.  dX may be
 * dY, dS or V (same pointer and leading dimension).
 */
int sgemm_rmsnorm_backward(int type, int M, int K,
                           const void *dY, int lddy,
                           const void *V, int ldv,
                           const void *w, float eps,
                           const void *dS, int ldds,
                           void *dX, int lddx,
                           void *dw,
                           sgemm_stream_t stream);

/*
 * sgemm_linear8 -- a projection of rows in 8 bits by a weight in 8 bits with a scale for each
 * output column:
 *
 *   Y[i][j] = scale[i] * wscale[j] * (sum over k of q[i][k] * W[k][j]) + bias[j]     (M x N)
 *
 * The rows are given as (q, scale) with X == NULL, or as the matrix X (M x K, of `type`), which the
 * call brings to rows of 8 bits itself.  W: K x N int8; wscale: N floats; bias: N elements of
 * `type`, or NULL.  Every int8 value, -128 too, counts as it stands.  The sums are exact, so K is at
 * most 131071 (SGEMM_ERR_TOO_LARGE); the rest is fp32, rounded once.  K == 0 gives bias, or 0.  Y
 * must not overlap an input.
 */
int sgemm_linear8(int type, int M, int N, int K,
                  const void *X, int ldx,
                  const signed char *q, int ldq, const float *scale,
                  const signed char *W, int ldw, const float *wscale,
                  const void *bias,
                  void *Y, int ldy,
                  sgemm_stream_t stream);

/* ------------------------------------------------------------------ gated block
 *
 * Two projections of the same rows, an activation of the one and its product with the other: the
 * feed-forward block of a language model up to its last projection.  `act`: sgemm_act of sgemm.h,
 * SGEMM_ACT_SILU among them.  SILU and GELU are +inf at +inf and NaN at -inf, as their formulas
 * are.
 */

/*
 * sgemm_gated -- forward, for one token up to a long prefill:
 *
 *   G = X * Wg,  U = X * Wu,  H = act(G) * U                (M x N each)
 *
 * X: M x K; Wg, Wu: K x N.  G and U, NULL together, receive the projections for the backward pass;
 * H is made of their fp32 sums, before they are rounded to `type`.  K == 0 gives zero sums.
 * The outputs must not overlap an input or each other.
 */
int sgemm_gated(int type, int M, int N, int K,
                const void *X, int ldx,
                const void *Wg, int ldwg,
                const void *Wu, int ldwu,
                int act,
                void *G, int ldg,
                void *U, int ldu,
                void *H, int ldh,
                sgemm_stream_t stream);

/*
 * sgemm_gated_backward -- the gradients of sgemm_gated for dH (M x N), given X, G and U:
 *
 *   dG = dH * U * act'(G),  dU = dH * act(G)
 *   dX = dG * Wg^T + dU * Wu^T                              (M x K)
 *   dWg = X^T * dG,  dWu = X^T * dU                         (K x N each)
 *
 * relu'(0) is 0.  In bfloat16 dG and dU are rounded to bfloat16 before the products that take them.
 * dX may be NULL (Wg and Wu are then not read), and dWg and dWu together (X is then not read).
 * M == 0 or N == 0 gives zeros.  The outputs must not overlap an input or each other.
 */
int sgemm_gated_backward(int type, int M, int N, int K, int act,
                         const void *dH, int lddh,
                         const void *X, int ldx,
                         const void *G, int ldg,
                         const void *U, int ldu,
                         const void *Wg, int ldwg,
                         const void *Wu, int ldwu,
                         void *dX, int lddx,
                         void *dWg, int lddwg,
                         void *dWu, int lddwu,
                         sgemm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_FP32_GEMM_02_GB300_SGEMM_LAYERS_H */
