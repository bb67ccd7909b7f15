// host_state.h -- the library's per-process and per-device state as the
// translation units beside sgemm.cu use it (sgemm.cu holds and defines it).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstddef>
#include <cstdint>

namespace sgh {

// SM count and workspace pool of the current device, or a status other than
// SGEMM_OK (first use sets the device's state up).
int current_device(int *sm_count, cudaMemPool_t *pool);

// Records a failed CUDA call (sgemm_last_cuda_error) and returns its status.
int cuda_fail(cudaError_t e);

// The same for a driver call's result.
int driver_fail(int result);

// cuTensorMapEncodeTiled, after current_device().
PFN_cuTensorMapEncodeTiled_v12000 encode_tiled();

// A launch for sgemm_kernel_launch_count(); `main_kernel`, where it is not
// null, becomes the calling thread's sgemm_last_kernel().
void count_launch(const char *main_kernel = nullptr);

// The limit of in-kernel waits (sgemm_set_wait_timeout_ns).
unsigned long long wait_timeout_ns();

// Reads, and clears where asked, the copies of the device error word of act8.cu, lora.cu and
// parts_gemm.cu.
cudaError_t act8_error_word(unsigned *v, bool clear);
cudaError_t lora_error_word(unsigned *v, bool clear);
cudaError_t parts_gemm_error_word(unsigned *v, bool clear);

// Largest size that an entry point accepts.
constexpr int kMaxDim = 0x7fffffff - 0xffff;

// A launch that need not wait for the kernel before it on the stream (programmatic stream
// serialization): its blocks start once every block of that one has called
// sg::launch_dependents() or ended, and sg::wait_prerequisites() waits for that one's end.  It
// saves the launch's latency between two kernels.  What makes it safe:
//  1. The first kernel of a call is launched plainly, or waits before it calls
//     launch_dependents().  So all work enqueued before the call has ended when its second kernel
//     starts, and a later kernel may at once read the caller's inputs and write workspace that no
//     kernel of this call has used yet.  (A call to launch_dependents() above that wait would be a
//     race with the call before.)
//  2. What another kernel of the call writes, or still reads, is touched after the wait only.
//  3. A kernel whose blocks do not all wait has its first block wait at the end: its own end then
//     says that the kernels before it have ended, which is what the next one's wait relies on.
// Kernels that make use of 1: parts_kernel beside the grouping, few_rows_rank_kernel beside the
// product, and few_rows_finish_kernel, which reads ids, B and bias before its wait.
template <class... P, class... Args>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                         const Args &...args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// Workspace of one call: `bytes` from the device's pool, handed out in
// 256-byte aligned pieces, given back to it on `stream` at the end of the call.
class Workspace {
public:
    Workspace(cudaMemPool_t pool, cudaStream_t stream) : pool_(pool), stream_(stream) {}
    ~Workspace() { release(); }
    Workspace(const Workspace &) = delete;
    Workspace &operator=(const Workspace &) = delete;

    static constexpr size_t piece(size_t bytes) { return (bytes + 255) & ~size_t(255); }

    int allocate(size_t bytes);
    template <class T>
    T *take(size_t count) {
        T *p = reinterpret_cast<T *>(base_ + used_);
        used_ += piece(count * sizeof(T));
        return p;
    }
    int release();

private:
    cudaMemPool_t pool_;
    cudaStream_t stream_;
    char *base_ = nullptr;
    size_t used_ = 0;
};

}  // namespace sgh
