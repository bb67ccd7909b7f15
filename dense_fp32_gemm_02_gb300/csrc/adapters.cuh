// adapters.cuh -- the adapters of a call as the kernels see them.
#pragma once

#include "elements.cuh"

namespace sgl {

// bfloat16 parts of the rank side's fp32 sums: all of their 24 bits, whatever the call's type.
// (Two, 16 bits, would do for most of a bfloat16 result, but not where the sums cancel.  4096 x
// 4096 x 4096 bfloat16, rank 32 of 4, us: backward 155 with two and 165 with three, of it the stack's
// gradients 60 and 67; forward 118 and 120.)
constexpr int S_PARTS = 3;

// The adapters of a call: which one a row uses, its rank and scale.
struct Adapters {
    const int *ids, *ranks;
    const float *scales;
    int L, R;

    __device__ int of_row(long long i) const {
        const int a = L > 0 ? ids[i] : -1;
        return unsigned(a) < unsigned(L) ? a : -1;
    }
    __device__ int rank(int a) const { return ranks ? min(max(ranks[a], 0), R) : R; }
    __device__ float scale(int a) const { return scales ? scales[a] : 1.0f; }
};

// A stack of L matrices.
template <class T>
struct Stack {
    T *p;
    long long ld, stride;

    __device__ T *matrix(int a) const { return p + a * stride; }
};

}  // namespace sgl
