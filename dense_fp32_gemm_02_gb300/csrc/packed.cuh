// packed.cuh -- a matrix as an operand of the tensor cores' products: itself, where the TMA can
// read it, or its parts in the workspace.
#pragma once

#include "host_state.h"
#include "lora.cuh"
#include "parts_gemm.h"

namespace sgl {

using sgh::aligned;

inline long long pitch8(long long cols) { return (cols + 7) / 8 * 8; }

// A matrix that the TMA reads where it lies: bfloat16, 16-byte aligned rows.
template <class T>
bool in_place(const T *p, int ld) {
    return sizeof(T) == 2 && aligned(p, 16) && ld % 8 == 0;
}

template <class T>
bool wide_rows(const T *p, long long ld) {
    return aligned(p, 16) && ld % (16 / (long long)sizeof(T)) == 0;
}

// The parts of a rows x cols matrix as an operand: the matrix itself, or planes in the
// workspace that parts_kernel fills.
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
    PartsJob<Rows<T>> job() const {   // (no rows where the TMA reads the matrix itself)
        return PartsJob<Rows<T>>(Rows<T>{src, ld}, direct ? 0 : int(rows), int(cols), wide_rows(src, ld), parts);
    }
    sgp::Operand operand() const {
        if (direct)
            return {reinterpret_cast<const bf16 *>(src), cols, rows, 1, ld, rows * (long long)ld};
        return {parts.p, cols, rows, PARTS, pitch, rows * pitch};
    }
};

}  // namespace sgl
