// parts_gemm.cu -- launches of parts_gemm.cuh: tensor maps, the split of the
// contraction, and the kernels of the three layouts in both types.
#include "../../include/sgemm_layers.h"

#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "host_state.h"
#include "parts_gemm.cuh"
#include "variant.cuh"

namespace {

using namespace sgp;

template <class T, Layout LAYOUT>
struct Kernel {
    static constexpr bool F32 = sizeof(T) == 4, A_MN = LAYOUT == WEIGHT_GRAD, B_MN = LAYOUT != INPUT_GRAD;
    static constexpr int PA = F32 && LAYOUT != WEIGHT_GRAD ? 3 : 1, PB = F32 ? 3 : 1;
    static constexpr auto *main = &parts_gemm_kernel<T, PA, PB, A_MN, B_MN, LAYOUT == INPUT_GRAD, false, false>;
    // (of several parts the one kernel is for any length)
    static constexpr auto *main_long = &parts_gemm_kernel<T, PA, PB, A_MN, B_MN, LAYOUT == INPUT_GRAD, false, PA * PB == 1>;
    static cudaError_t set_attr() {
        const cudaError_t e = cudaFuncSetAttribute(main, cudaFuncAttributeMaxDynamicSharedMemorySize, int(SMEM_BYTES));
        if (e != cudaSuccess) return e;
        return cudaFuncSetAttribute(main_long, cudaFuncAttributeMaxDynamicSharedMemorySize, int(SMEM_BYTES));
    }
};

template <class T>
struct RankKernel {
    static constexpr int PARTS = sizeof(T) == 4 ? 3 : 1;
    static constexpr auto *main = &parts_gemm_kernel<T, PARTS, PARTS, false, false, false, true, false>;
    static cudaError_t set_attr() {
        return cudaFuncSetAttribute(main, cudaFuncAttributeMaxDynamicSharedMemorySize, int(SMEM_BYTES));
    }
};

}  // namespace

int sgp::encode(CUtensorMap *map, const Operand &o, uint32_t box_inner, uint32_t box_outer) {
    const cuuint64_t dims[3] = {cuuint64_t(o.inner), cuuint64_t(o.outer), cuuint64_t(o.planes)};
    const cuuint64_t strides[2] = {cuuint64_t(o.pitch) * 2, cuuint64_t(o.plane_pitch) * 2};
    const cuuint32_t box[3] = {box_inner, box_outer, 1}, steps[3] = {1, 1, 1};
    const CUresult r = sgh::encode_tiled()(
        map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<bf16 *>(o.p), dims, strides, box, steps,
        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SGEMM_OK : sgh::driver_fail(int(r));
}

cudaError_t sgh::parts_gemm_error_word(unsigned *v, bool clear) { return sgv::unit_error_word(v, clear); }

int sgp::set_up() {
    static std::atomic<unsigned long long> done{0};   // a bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return sgh::cuda_fail(e);
    if (done.load() >> dev & 1) return SGEMM_OK;
    cudaError_t (*const all[])() = {
        &Kernel<float, FORWARD>::set_attr, &Kernel<bf16, FORWARD>::set_attr,
        &Kernel<float, INPUT_GRAD>::set_attr, &Kernel<bf16, INPUT_GRAD>::set_attr,
        &Kernel<float, WEIGHT_GRAD>::set_attr, &Kernel<bf16, WEIGHT_GRAD>::set_attr,
        &RankKernel<float>::set_attr, &RankKernel<bf16>::set_attr};
    for (auto set : all)
        if ((e = set()) != cudaSuccess) return sgh::cuda_fail(e);
    done.fetch_or(1ull << dev);
    return SGEMM_OK;
}

// In units of one part pair's slab (64 k of a 256 x 256 tile, 0.27 us on a pair): a
// wave takes its slabs, about 8 units of pipeline fill and epilogue; partial sums
// are written and read once at about 5 TB/s, by a second launch (12 units).  A last wave
// of half-width tiles counts half after others, as narrow tiles where it is the only one.
//
// Tiles of 128 to 224 columns fill the pairs better where there are few.  With several
// products to a slab one takes 1.1 times its share of a slab's time, and not less than
// 0.57 units for each part that it loads; bfloat16's one product is bound by its loads,
// which do not get fewer, so narrow tiles gain nothing there (128 columns: 8192 x 4096 x
// 4096 in 332 us for 208).
//
// The least estimate over the widths and up to 64 ranges: 64 x 4096 x 4096 bfloat16
// takes 4 ranges (18 us; 1: 26, 2: 21, 8: 22), 512 rows 1 (27; 2: 29, 4: 34); the float32
// weight gradient 4097 x 1023 x 3001 tiles of 160 columns (the call 82.5 us; 256: 93.3, 224:
// 89.1, 192: 84.1, 128: 128.8), the input gradient 3001 x 1024 x 1023 of 192 (75.4; 256:
// 81.8).  120 float32 products of random sizes take 0.966 of the time that 256 columns
// take, the best width of each 0.954.
Split sgp::plan_split(int M, int N, int K, int products, int sms, Outputs outputs, int contractions) {
    const long long pairs = std::max(1, sms / 2);
    const long long slabs = contractions * ((K + BK - 1LL) / BK), columns = N * (outputs == ALONE ? 1LL : 2LL);
    const int parts = products == 1 ? 2 : products == 3 ? 4 : 6;   // that a slab loads
    auto slab_cost = [&](int width) {
        return width == TILE || products == 1 ? double(products)
                                              : std::max(1.1 * products * width / TILE, 0.57 * parts);
    };
    Split best{1, TILE, 0};
    double least = 0;
    for (int width = TILE; width >= (products == 1 ? TILE : TILE / 2);
         width -= outputs == HALF_EACH ? 64 : 32) {
        const long long across = outputs == ONE_BY_ONE ? 2 * ((N + width - 1LL) / width) : (columns + width - 1) / width;
        const long long tiles = ((M + 255LL) / 256) * across;
        for (long long s = 1; s <= std::min(64LL, std::max(1LL, slabs)); ++s) {
            const long long per = (slabs + s - 1) / s;
            if ((slabs + per - 1) / per != s) continue;      // a range would be empty
            const long long items = tiles * s, waves = items / pairs, rest = items % pairs;
            const bool halves = width == TILE && s == 1 && 2 * rest <= pairs;   // the last wave's
            const double last = rest == 0 ? 0.0 : halves && waves > 0 ? 0.5 : 1.0;
            const double slab = slab_cost(halves && waves == 0 ? TILE / 2 : width);
            const double cost = (double(waves) + last) * (double(per) * slab + 8.0) +
                                (s > 1 ? 12.0 + double(s) * M * columns * 8.0 / 5.0e6 / 0.27 : 0.0);
            if (least == 0 || cost < least) {
                least = cost;
                best = Split{int(s), width, s > 1 ? size_t(s) * M * size_t(columns) : 0};
            }
        }
    }
    return best;
}

template <class T, bool TRANS>
int sgp::finish(int M, int N, int splits, const float *partial, const int4 *planes,
                const Epilogue<T, TRANS> &epi, cudaStream_t stream) {
    // grid rows are at most 65535 to a launch
    for (long long r = 0; r < M; r += 65535) {
        const int rows = int(std::min<long long>(65535, M - r));
        Epilogue<T, TRANS> at = epi;
        at.ad.ids += at.ad.L > 0 ? r : 0;
        at.S += r * at.lds;
        at.out += r * at.ldo;
        cudaError_t e = sgh::launch_early(finish_kernel<T, TRANS>, dim3(unsigned((N + 255) / 256), unsigned(rows)), 256, 0,
                                          stream, M, N, splits, partial + r * N, planes, int(r), at);
        if (e != cudaSuccess) return sgh::cuda_fail(e);
        sgh::count_launch();
        e = cudaGetLastError();
        if (e != cudaSuccess) return sgh::cuda_fail(e);
    }
    return SGEMM_OK;
}

template <class T, Layout LAYOUT>
int sgp::run(const Product &p, const Epilogue<T, LAYOUT == INPUT_GRAD> &epi, Split split,
             float *partial, int sms, cudaStream_t stream, Mode mode) {
    using K = Kernel<T, LAYOUT>;
    int st = set_up();
    if (st != SGEMM_OK) return st;
    const long long tiles_m = (p.M + TILE - 1LL) / TILE, tiles_n = (p.N + split.tile_n - 1LL) / split.tile_n;
    if (tiles_m * tiles_n * split.splits > (1LL << 30)) return SGEMM_ERR_TOO_LARGE;
    KernelParams kp{};
    kp.M = p.M;
    kp.N = p.N;
    kp.tiles_m = int(tiles_m);
    kp.tiles_n = int(tiles_n);
    kp.tile_n = split.tile_n;
    kp.group_m = 8;
    kp.slabs = int((p.K + BK - 1LL) / BK);
    kp.splits = split.splits;
    kp.per_split = (kp.slabs + split.splits - 1) / split.splits;
    kp.partial = partial;
    kp.timeout_ns = sgh::wait_timeout_ns();
    CUtensorMap mA, mB, mH, mV;
    if ((st = encode(&mA, p.a, BK, K::A_MN ? BK : ROWS)) != SGEMM_OK ||
        (st = encode(&mB, p.b, BK, K::B_MN ? BK : ROWS)) != SGEMM_OK)
        return st;
    mH = mA;
    mV = mB;
    if (p.planes) {
        kp.planes = p.planes;
        kp.plane_adapter = p.plane_adapter;
        kp.most_planes = p.most_planes;
        kp.capacity = p.capacity;
        kp.width = p.width;
        kp.L = epi.ad.L;
        if ((st = encode(&mH, p.h, BK, ROWS)) != SGEMM_OK ||
            (st = encode(&mV, p.v, BK, uint32_t(std::min(p.width, BK)))) != SGEMM_OK)
            return st;
    }
    const long long pairs = std::min<long long>(tiles_m * tiles_n * split.splits * (split.splits == 1 ? 2 : 1),
                                                std::max(1, sms / 2));
    cudaError_t e = sgh::launch_early(kp.per_split > LONG_CHUNK ? K::main_long : K::main, dim3(unsigned(2 * pairs)), THREADS,
                                      SMEM_BYTES, stream, mA, mB, mH, mV, kp, epi);
    if (e != cudaSuccess) return sgh::cuda_fail(e);
    sgh::count_launch(K::F32 ? "bf16 parts of float32, tcgen05 cta_group::2, pair tiles of 256 rows"
                             : "bf16, tcgen05 cta_group::2, 256x256 pair tiles");
    e = cudaGetLastError();
    if (e != cudaSuccess) return sgh::cuda_fail(e);
    if (split.splits > 1 && mode == WHOLE)
        return finish<T, LAYOUT == INPUT_GRAD>(p.M, p.N, split.splits, partial, p.planes, epi, stream);
    return SGEMM_OK;
}

// Ranges of the rank side's contraction: the count whose waves of (256 rows, range) items
// over the pairs take the fewest slabs, with six for filling and emptying.
int sgp::rank_splits(int M, int K, int sms) {
    const long long pairs = std::max(1, sms / 2), tiles = (M + 255LL) / 256, slabs = (K + BK - 1LL) / BK;
    int best = 1;
    long long least = 0;
    for (long long n = 1; n <= std::min(64LL, slabs); ++n) {
        const long long per = (slabs + n - 1) / n;
        if ((slabs + per - 1) / per != n) continue;   // a range would be empty
        const long long cost = ((tiles * n + pairs - 1) / pairs) * (per + 6);
        if (n == 1 || cost < least) least = cost, best = int(n);
    }
    return best;
}

template <class T>
int sgp::run_rank(const RankProduct &p, int splits, float *partial, int sms, cudaStream_t stream) {
    using K = RankKernel<T>;
    int st = set_up();
    if (st != SGEMM_OK) return st;
    const long long tiles_m = (p.M + TILE - 1LL) / TILE, groups = (p.most_planes + 3LL) / 4;
    const long long items = tiles_m * groups * splits;
    if (items > (1LL << 30)) return SGEMM_ERR_TOO_LARGE;
    KernelParams kp{};
    kp.M = p.M;
    kp.N = int(groups * TILE);
    kp.tiles_m = int(tiles_m);
    kp.tiles_n = int(groups);
    kp.tile_n = TILE;
    kp.group_m = 8;
    kp.slabs = int((p.K + BK - 1LL) / BK);
    kp.splits = splits;
    kp.per_split = (kp.slabs + splits - 1) / splits;
    kp.planes = p.planes;
    kp.plane_adapter = p.plane_adapter;
    kp.position = p.position;
    kp.most_planes = p.most_planes;
    kp.width = p.width;
    kp.L = p.ad.L;
    kp.partial = partial;
    kp.timeout_ns = sgh::wait_timeout_ns();
    CUtensorMap mA, mB;
    if ((st = encode(&mA, p.x, BK, ROWS)) != SGEMM_OK ||
        (st = encode(&mB, p.v, BK, uint32_t(std::min(p.width, 32)))) != SGEMM_OK)
        return st;
    Epilogue<T, false> epi{};
    epi.ad = p.ad;
    const long long pairs = std::min<long long>(items, std::max(1, sms / 2));
    const cudaError_t e = sgh::launch_early(K::main, dim3(unsigned(2 * pairs)), THREADS, SMEM_BYTES, stream, mA, mB, mA, mB,
                                            kp, epi);
    if (e != cudaSuccess) return sgh::cuda_fail(e);
    sgh::count_launch();
    const cudaError_t after = cudaGetLastError();
    return after == cudaSuccess ? SGEMM_OK : sgh::cuda_fail(after);
}

namespace sgp {
#define LAYER_PRODUCT(T, LAYOUT)                                                                  \
    template int run<T, LAYOUT>(const Product &, const Epilogue<T, LAYOUT == INPUT_GRAD> &, Split, \
                                float *, int, cudaStream_t, Mode)
LAYER_PRODUCT(float, FORWARD);
LAYER_PRODUCT(bf16, FORWARD);
LAYER_PRODUCT(float, INPUT_GRAD);
LAYER_PRODUCT(bf16, INPUT_GRAD);
LAYER_PRODUCT(float, WEIGHT_GRAD);
LAYER_PRODUCT(bf16, WEIGHT_GRAD);
#undef LAYER_PRODUCT
#define LAYER_FINISH(T, TRANS) \
    template int finish<T, TRANS>(int, int, int, const float *, const int4 *,                    \
                                  const Epilogue<T, TRANS> &, cudaStream_t)
LAYER_FINISH(float, false);
LAYER_FINISH(bf16, false);
LAYER_FINISH(float, true);
LAYER_FINISH(bf16, true);
#undef LAYER_FINISH
template int run_rank<float>(const RankProduct &, int, float *, int, cudaStream_t);
template int run_rank<bf16>(const RankProduct &, int, float *, int, cudaStream_t);
}  // namespace sgp
