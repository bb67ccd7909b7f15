// parts_gemm.h -- products of matrices given as sums of bfloat16 parts, on the
// tensor cores (parts_gemm.cu), as the layer entry points call them.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "adapters.cuh"

namespace sgp {

// One operand: `parts` planes of bfloat16 that add up to the matrix, row-major
// (inner: the contiguous dimension), the pitch and the plane pitch multiples of 8
// elements and the address of 16 bytes.
struct Operand {
    const sgl::bf16 *p = nullptr;
    long long inner = 0, outer = 0, planes = 0, pitch = 0, plane_pitch = 0;
};

// What becomes of an output element, fp32 up to its one rounding:
//   out = sum + sum_r S[i][r] * V_a(i)[r][j] + bias[j] + beta * out
// S is M x R (its scale in it), V the caller's own stack (TRANS: stored N x R).
template <class T, bool TRANS>
struct Epilogue {
    sgl::Adapters ad;
    const float *S;
    long long lds;
    sgl::Stack<const T> V;
    const T *bias;
    float beta;
    T *out;
    long long ldo;
};

// out (M x N) = a * b over a contraction K.  a is M x K stored K-major (inner = K) or
// M-major (inner = M), b likewise.  The rank-side term joins the product as more of its
// contraction, 64 columns at a time: `h` the planes of 256 x 64 that sgl::Groups
// describes (part * capacity + plane), `v` the adapters' parts (part * L + a, `width` x
// N).  A tile whose planes may not be used gets the term by FMAs from S and the caller's
// stack.
struct Product {
    int M, N, K;
    Operand a, b, h, v;
    const int4 *planes = nullptr;
    const int4 *plane_adapter = nullptr;
    int most_planes = 0, capacity = 0, width = 64;
};

// The rank side's own product: S before its scale.  `x` the parts of X (M x K, K-major),
// `v` those of the stack with K along its rows (plane part * L + a, width x K).  A row's
// sums over each range go to partial[range][row][width].
struct RankProduct {
    int M, K, width, most_planes;   // planes of a tile at most
    Operand x, v;
    sgl::Adapters ad;
    const int4 *planes;
    const int4 *plane_adapter;
    const int *position;
};
int rank_splits(int M, int K, int sms);
template <class T>
int run_rank(const RankProduct &p, int splits, float *partial, int sms, cudaStream_t stream);

enum Layout { FORWARD, INPUT_GRAD, WEIGHT_GRAD };   // (a, b): (K, N)-major, (K, K), (M, N)

// How the contraction is split over the SMs: `splits` ranges whose fp32 partial sums
// (partial_floats of them) a second kernel adds in order, or one.
struct Split {
    int splits, tile_n;   // tile_n: columns of a tile
    size_t partial_floats;
};
// `outputs`: one matrix, or two of N columns each whose tiles are one list (ONE_BY_ONE) or hold
// half their columns of either (HALF_EACH); `contractions` of K each.
enum Outputs { ALONE, ONE_BY_ONE, HALF_EACH };
Split plan_split(int M, int N, int K, int products, int sms, Outputs outputs = ALONE, int contractions = 1);

// The tensor map of an operand with boxes of box_inner x box_outer elements of one plane.
int encode(CUtensorMap *map, const Operand &o, uint32_t box_inner, uint32_t box_outer);

// float: a of 3 parts (1 in WEIGHT_GRAD) and b of 3; bfloat16: one part each.
// The kernel is launched early (host_state.h).  PARTIALS leaves the partial sums (of one
// range too) to the caller.
enum Mode { WHOLE, PARTIALS };
template <class T, Layout LAYOUT>
int run(const Product &p, const Epilogue<T, LAYOUT == INPUT_GRAD> &epi, Split split, float *partial,
        int sms, cudaStream_t stream, Mode mode = WHOLE);

// The second kernel alone: out from `splits` partial sums (none: the epilogue of zero).
// Rows of tiles that have planes already have their rank-side term (planes null: none).
template <class T, bool TRANS>
int finish(int M, int N, int splits, const float *partial, const int4 *planes, const Epilogue<T, TRANS> &epi,
           cudaStream_t stream);

int set_up();   // the kernels' attributes on the current device (its first call)

}  // namespace sgp
