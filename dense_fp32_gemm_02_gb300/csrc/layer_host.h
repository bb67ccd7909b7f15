// layer_host.h -- argument checks and launches that the units of the layer's entry points share.
#pragma once

#include <algorithm>

#include "../../include/sgemm_layers.h"
#include "host_state.h"

namespace sgh {

// A matrix that an entry point refuses: none, not aligned to its elements, or with overlapping rows.
inline bool bad_matrix(const void *p, int ld, int columns, size_t element) {
    return !p || !aligned(p, element) || ld < std::max(1, columns);
}
// The same of one that may be left out, and of vectors.
inline bool bad_optional(const void *p, int ld, int columns, size_t element) {
    return p && bad_matrix(p, ld, columns, element);
}
inline bool bad_vector(const void *p, size_t element) { return !p || !aligned(p, element); }

inline size_t element_bytes(int type) { return type == SGEMM_BF16 ? 2 : 4; }

inline int check_sizes(int type, std::initializer_list<int> sizes) {
    if (type != SGEMM_F32 && type != SGEMM_BF16) return SGEMM_ERR_INVALID_ARG;
    for (int n : sizes)
        if (n < 0) return SGEMM_ERR_INVALID_ARG;
    for (int n : sizes)
        if (n > kMaxDim) return SGEMM_ERR_TOO_LARGE;
    return SGEMM_OK;
}

// Rows that can be read or written 16 bytes at a time (or that there are none of).
template <class T>
bool wide_rows(const T *p, long long ld) {
    return !p || (aligned(p, 16) && ld % (16 / (long long)sizeof(T)) == 0);
}

// Counts a launch that returned `e`, where it was made, and returns its status.
inline int launched(cudaError_t e, const char *main_kernel) {
    if (e != cudaSuccess) return cuda_fail(e);
    count_launch(main_kernel);
    return SGEMM_OK;
}

// An early launch (host_state.h), counted.
template <class... P, class... Args>
int launch(const char *text, void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
           const Args &...args) {
    return launched(launch_early(kernel, grid, threads, smem, stream, args...), text);
}

// The same in clusters of `cluster` blocks.
template <class... P, class... Args>
int launch_cluster(const char *text, void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, int cluster, cudaStream_t stream,
                   const Args &...args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster), attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return launched(cudaLaunchKernelEx(&cfg, kernel, P(args)...), text);
}

// Rows in 8 bits, each with a scale (norm.cu): q and scale of the rows of X.
int rows8(int type, int M, int K, const void *X, int ldx, signed char *q, long long ldq, float *scale, int sms,
          cudaStream_t stream);

}  // namespace sgh
