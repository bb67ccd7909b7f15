// gated.cuh -- kernels of the gated block beside its products on the tensor cores (pair_gemm.cuh):
// few rows, the sums of a split contraction, and the gradients of G and U.
//
//   H = act(G) * U,  G = X Wg,  U = X Wu;   dG = dH U act'(G),  dU = dH act(G)
#pragma once

#include "gate.cuh"
#include "rows.cuh"

namespace sgl {

// ------------------------------------------------------------------ few rows of float32
// Bound by reading both matrices once.  The products of rows.cuh, the blocks of Wg's and then of
// Wu's in one launch; their sums over each range go to partial[range][row][column], U's behind G's.
template <int MR, bool WIDE>
__global__ void __launch_bounds__(RANK_THREADS, stream_blocks(MR))
    gated_stream_kernel(RowsWork w, Rows<float> X, const float *Wg, long long ldg, const float *Wu, long long ldu) {
    __shared__ __align__(16) float sm[StreamRows<float, MR>::FLOATS];
    sg::wait_prerequisites();
    sg::launch_dependents();
    const int n = w.across * w.ranges, second = int(blockIdx.x) >= n;
    if (!SG_IN_RANGE(int(blockIdx.x) < 2 * n)) return;
    stream_rows<float, MR, WIDE>(w, int(blockIdx.x) - second * n, X, second ? Wu : Wg, second ? ldu : ldg,
                             w.partial + second * (long long)w.ranges * w.M * w.N, sm);
}

static __global__ void __launch_bounds__(RANK_THREADS, 2)
    gated_few_rows_kernel(RowsWork w, Rows<float> X, const float *Wg, long long ldg, const float *Wu, long long ldu,
                          bool w_wide) {
    extern __shared__ __align__(16) unsigned char smem_rows[];
    sg::wait_prerequisites();
    sg::launch_dependents();
    const int n = w.across * w.ranges, second = int(blockIdx.x) >= n;
    if (!SG_IN_RANGE(int(blockIdx.x) < 2 * n)) return;
    few_rows<1>(w, int(blockIdx.x) - second * n, X, second ? Wu : Wg, second ? ldu : ldg, w_wide,
                 w.partial + second * (long long)w.ranges * w.M * w.N, smem_rows);
}

// ------------------------------------------------------------------ sums of ranges
// x and y from `ranges` partial sums each, added in order: the block's outputs, or (GATED false) the
// two of a product of two.  A thread to four columns of a row, grid rows to the rows.
template <class T>
struct PairOut {
    T *out, *out1, *H;   // G and U (or none) and H; or the two outputs
    long long ldo, ldo1, ldh;
    int act;
};
template <class T, bool GATED>
__global__ void __launch_bounds__(128)
    pair_finish_kernel(int M, int N, int ranges, const float *__restrict__ px, const float *__restrict__ py,
                       long long pitch, long long plane, bool wide, PairOut<T> to) {
    const int j = (blockIdx.x * 128 + threadIdx.x) * 4, n = min(4, N - j);
    for (long long i = blockIdx.y; i < M; i += gridDim.y) {
        if (j >= N || !SG_IN_RANGE(pitch >= N)) break;
        if (i == blockIdx.y) sg::wait_prerequisites();
        float x[4] = {}, y[4] = {};
        const float *gx = px + i * pitch + j, *gy = py + i * pitch + j;
#pragma unroll 4
        for (int r = 0; r < ranges; ++r) {
            float a[4], b[4];
            if (wide) {
                load4(gx + r * plane, a);
                load4(gy + r * plane, b);
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d) a[d] = d < n ? gx[r * plane + d] : 0.0f, b[d] = d < n ? gy[r * plane + d] : 0.0f;
            }
#pragma unroll
            for (int d = 0; d < 4; ++d) x[d] += a[d], y[d] += b[d];
        }
        auto write = [&](T *p, const float (&v)[4]) {
#pragma unroll
            for (int d = 0; d < 4; ++d)
                if (d < n) p[d] = from_f32<T>(v[d]);
        };
        if (to.out) {
            write(to.out + i * to.ldo + j, x);
            write(to.out1 + i * to.ldo1 + j, y);
        }
        if constexpr (GATED) {
            float h[4];
            with_act(to.act, [&](auto act) {
#pragma unroll
                for (int d = 0; d < 4; d += 2) {
                    const float2 v = gate_value<T, decltype(act)::value>(make_float2(x[d], x[d + 1]));
                    h[d] = v.x * y[d], h[d + 1] = v.y * y[d + 1];
                }
            });
            write(to.H + i * to.ldh + j, h);
        }
    }
}

// ------------------------------------------------------------------ gradients of G and U
// dG and dU as operands of the products that take them: bfloat16, rounded to nearest as every
// other operand of these products is held, or the three parts of float32, exactly.  The rounding is
// 2^-8 of a term at most, of random sign, beside the same of an output's own (4096 x 4096 x 8192:
// gradients 2.35e-3 from 64 bits in the 2-norm, where the outputs' rounding alone leaves 1.66e-3; two
// bfloat16 to a value would make the products, 690 of 740 us, twice as long).  A thread to eight
// columns of a row; bound by its bytes.
template <class T>
struct SlopesJob {
    const T *dH, *G, *U;
    long long ldh, ldg, ldu;
    int M, N, act;
    bool wide;
    Parts dG, dU;
    Divisor per_row;   // octets
};

template <class T>
__device__ __forceinline__ void store_operand(const Parts &to, long long row, long long col, const float (&x)[8]) {
    if constexpr (sizeof(T) == 4)
        store_parts<3>(to, row, col, x);
    else
        store8(to.p + row * to.pitch + col, x);
}

template <class T, int ACT>
__device__ __forceinline__ void take_slopes(const SlopesJob<T> &a) {
    const long long total = (long long)a.M * a.per_row.d, step = (long long)gridDim.x * 256;
    const bool small = total <= 0x7fffffffll;
    for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < total; t += step) {
        const long long i = small ? (long long)a.per_row.quotient(unsigned(t)) : t / a.per_row.d;
        const int c = int(t - i * a.per_row.d) * 8;
        if (!SG_IN_RANGE(i < a.M && c < a.N && c + 8 <= a.dG.pitch && (i + 1) * a.dG.pitch <= a.dG.plane)) continue;
        float dh[8], g[8], u[8], dg[8], du[8];
        const T *ph = a.dH + i * a.ldh + c, *pg = a.G + i * a.ldg + c, *pu = a.U + i * a.ldu + c;
        if (a.wide && c + 8 <= a.N) {
            load8(ph, dh);
            load8(pg, g);
            load8(pu, u);
        } else if (c + 8 > a.N || !load8_shifted(ph, a.dH, a.dH + (a.M - 1) * a.ldh + a.N, dh) ||
                   !load8_shifted(pg, a.G, a.G + (a.M - 1) * a.ldg + a.N, g) ||
                   !load8_shifted(pu, a.U, a.U + (a.M - 1) * a.ldu + a.N, u)) {
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                const bool in = c + d < a.N;
                dh[d] = in ? to_f32(ph[d]) : 0.0f, g[d] = in ? to_f32(pg[d]) : 0.0f, u[d] = in ? to_f32(pu[d]) : 0.0f;
            }
        }
#pragma unroll
        for (int d = 0; d < 8; d += 2) {
            float2 value, rise;
            gate_both<T, ACT>(make_float2(g[d], g[d + 1]), value, rise);
            du[d] = dh[d] * value.x, du[d + 1] = dh[d + 1] * value.y;
            dg[d] = dh[d] * u[d] * rise.x, dg[d + 1] = dh[d + 1] * u[d + 1] * rise.y;
        }
        store_operand<T>(a.dG, i, c, dg);
        store_operand<T>(a.dU, i, c, du);
    }
}
template <class T>
__global__ void __launch_bounds__(256) gated_slopes_kernel(SlopesJob<T> a) {
    sg::wait_prerequisites();
    sg::launch_dependents();
    with_act(a.act, [&](auto act) { take_slopes<T, decltype(act)::value>(a); });
}

// ------------------------------------------------------------------ operands
// The parts of the operands that the TMA cannot read where they lie, in one launch (1025 x 1023 x 3001 in
// bfloat16 24.3 us, with X's in a launch of its own 25.9).  `beside`: not the call's first kernel, it runs beside the one before it.
template <class T>
__global__ void __launch_bounds__(256)
    gated_parts_kernel(PartsJob<Rows<T>> g, PartsJob<Rows<T>> u, PartsJob<Rows<T>> x, bool beside) {
    constexpr int PARTS = sizeof(T) == 4 ? 3 : 1;
    if (!beside) sg::wait_prerequisites();
    sg::launch_dependents();
    const long long t = (long long)blockIdx.x * 256 + threadIdx.x, step = (long long)gridDim.x * 256;
    take_parts<PARTS>(g, t, step);
    take_parts<PARTS>(u, t, step);
    take_parts<PARTS>(x, t, step);
    if (beside && blockIdx.x == 0) sg::wait_prerequisites();
}

}  // namespace sgl
