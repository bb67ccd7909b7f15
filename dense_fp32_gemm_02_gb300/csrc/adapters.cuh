// adapters.cuh -- the adapters of a call as the kernels see them.
#pragma once

#include "elements.cuh"

namespace sgl {

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
