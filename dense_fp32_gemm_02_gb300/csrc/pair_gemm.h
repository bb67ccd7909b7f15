// pair_gemm.h -- the products of the gated block and of 8-bit rows on the tensor cores
// (pair_gemm.cu), as their entry points call them.
#pragma once

#include <cuda_runtime.h>

#include "parts_gemm.h"

namespace sgq {

using sgl::bf16;

// What a product is of and what becomes of it (M rows, N columns of an output, a contraction K):
//   GATE  G = A B0, U = A B1:         H = act(G) * U, and G and U where they are wanted
//   SUM   A0 B0 + A1 B1:              out
//   TWO   A B0 and A B1:              out and out1
//   BYTES A B of int8 (as bfloat16):  out = scale_i * wscale_j * sum + bias_j
enum Mode { GATE, SUM, TWO, BYTES };

template <class T>
struct Output {
    T *out, *out1, *H;          // GATE: G, U (both or none) and H
    long long ldo, ldo1, ldh;
    int act;
    const float *scale, *wscale;
    const T *bias;
    const int *large;           // BYTES: whether sums of 2048 products may leave 2^24 (null: they may)
};

// Operands as in parts_gemm.h; SUM: the planes of `a` are A0's parts and then A1's; TWO: the
// planes of b[0] and b[1] are the parts of B0 and of B1.
struct Product {
    int M, N, K;
    sgp::Operand a, b[2];
};

// The split (sgp::Split) of a product: `columns` its outputs' columns taken together.
sgp::Split plan(Mode mode, int M, int N, int K, int products, int sms);

// float: three parts a side; bfloat16: one; BYTES: one (T is the output's type).  The kernel is
// launched early (host_state.h).  With several ranges the partial sums, splits x M x (columns of
// all outputs), are left to the caller's finishing kernel.
template <class T, Mode MODE>
int run(const Product &p, const Output<T> &out, sgp::Split split, float *partial, int sms, cudaStream_t stream);

}  // namespace sgq
