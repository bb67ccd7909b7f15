// pair_gemm.cu -- launches of pair_gemm.cuh: tensor maps, the split of the contraction, and the
// kernels of the four products.
#include "../../include/sgemm_layers.h"

#include <cudaTypedefs.h>

#include <algorithm>

#include "layer_host.h"
#include "pair_gemm.cuh"
#include "variant.cuh"

namespace {

using namespace sgq;

template <class T, Mode MODE>
struct Kernels {
    static constexpr bool A_MN = MODE == TWO, B_MN = MODE != SUM, BYTES_MODE = MODE == BYTES;
    static constexpr int PARTS = sizeof(T) == 4 && !BYTES_MODE ? 3 : 1;
    static constexpr auto *main = &pair_gemm_kernel<T, PARTS, A_MN, B_MN, MODE, false>;
    // (of several parts the one kernel is for any length)
    static constexpr auto *chunks = &pair_gemm_kernel<T, PARTS, A_MN, B_MN, MODE, PARTS == 1>;
};

}  // namespace

cudaError_t sgh::pair_gemm_error_word(unsigned *v, bool clear) { return sgv::unit_error_word(v, clear); }

sgp::Split sgq::plan(Mode mode, int M, int N, int K, int products, int sms) {
    return sgp::plan_split(M, N, K, products, sms, mode == GATE ? sgp::HALF_EACH : mode == TWO ? sgp::ONE_BY_ONE : sgp::ALONE,
                           mode == SUM ? 2 : 1);
}

template <class T, Mode MODE>
int sgq::run(const Product &g, const Output<T> &out, sgp::Split split, float *partial, int sms, cudaStream_t stream) {
    using K = Kernels<T, MODE>;
    Params p{};
    p.M = g.M, p.N = g.N;
    p.tiles_m = (g.M + TILE - 1) / TILE;
    p.tile_n = split.tile_n;
    const long long per = MODE == GATE ? split.tile_n / 2 : split.tile_n, across = (g.N + per - 1) / per;
    const long long tiles_n = MODE == TWO ? 2 * across : across;
    if (p.tiles_m * tiles_n * split.splits > (1LL << 30)) return SGEMM_ERR_TOO_LARGE;
    p.tiles_n = int(tiles_n);
    p.out_tiles = int(across);
    p.group_m = 8;
    p.first_slabs = (g.K + BK - 1) / BK;
    p.slabs = MODE == SUM ? 2 * p.first_slabs : p.first_slabs;
    p.splits = split.splits;
    p.per_split = (p.slabs + split.splits - 1) / split.splits;
    p.partial = partial;
    p.timeout_ns = sgh::wait_timeout_ns();
    const auto kernel = p.per_split > chunk_slabs(K::PARTS > 1, MODE == BYTES) ? K::chunks : K::main;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(SMEM_BYTES));
    if (e != cudaSuccess) return sgh::cuda_fail(e);
    // (a CTA's rows of A, the last ones of few left as they are in shared memory: they reach no output)
    const uint32_t a_rows = K::A_MN ? BK : uint32_t(std::min(ROWS, (g.M + 7) / 8 * 8));
    p.slab_bytes = uint32_t(K::PARTS) * (K::A_MN ? PART_BYTES : a_rows * BK * 2) + K::PARTS * PART_BYTES;
    CUtensorMap mA, mB0, mB1;
    int st;
    if ((st = sgp::encode(&mA, g.a, BK, a_rows)) != SGEMM_OK ||
        (st = sgp::encode(&mB0, g.b[0], BK, K::B_MN ? BK : ROWS)) != SGEMM_OK)
        return st;
    mB1 = mB0;
    if (MODE != BYTES && (st = sgp::encode(&mB1, g.b[1], BK, K::B_MN ? BK : ROWS)) != SGEMM_OK) return st;
    const long long items = p.tiles_m * tiles_n * split.splits;
    const long long pairs = std::min<long long>(items * (split.splits == 1 ? 2 : 1), std::max(1, sms / 2));
    return sgh::launch(MODE == BYTES         ? "int8 as bfloat16, tcgen05 cta_group::2, 256x256 pair tiles"
                       : K::PARTS > 1 ? "two products, bf16 parts of float32, tcgen05 cta_group::2"
                                      : "two products, bf16, tcgen05 cta_group::2, 256x256 pair tiles",
                       kernel, dim3(unsigned(2 * pairs)), THREADS, SMEM_BYTES, stream, mA, mB0, mB1, p, out);
}

namespace sgq {
#define PAIR_PRODUCT(T, MODE) \
    template int run<T, MODE>(const Product &, const Output<T> &, sgp::Split, float *, int, cudaStream_t)
PAIR_PRODUCT(float, GATE);
PAIR_PRODUCT(bf16, GATE);
PAIR_PRODUCT(float, SUM);
PAIR_PRODUCT(bf16, SUM);
PAIR_PRODUCT(float, TWO);
PAIR_PRODUCT(bf16, TWO);
PAIR_PRODUCT(float, BYTES);
PAIR_PRODUCT(bf16, BYTES);
#undef PAIR_PRODUCT
}  // namespace sgq
