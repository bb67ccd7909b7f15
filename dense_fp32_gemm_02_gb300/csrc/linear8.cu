// linear8.cu -- entry point of the product of int8 matrices with scales for each row and column.
#include <cstdlib>

#include "layer_host.h"
#include "byte_tiles.cuh"
#include "linear8.cuh"
#include "packed.cuh"
#include "pair_gemm.h"
#include "variant.cuh"

#define SGEMM_API extern "C" __attribute__((visibility("default")))

namespace {

using namespace sgl;

constexpr int kMostTerms = 131071;   // of 2^14 each at most: their sum stays under 2^31

struct Call {
    int type, M, N, K;
    const void *X;
    int ldx;
    const signed char *q;
    long long ldq;
    const float *scale;
    const signed char *W;
    int ldw;
    const float *wscale;
    const void *bias;
    void *Y;
    int ldy;
    cudaStream_t stream;
};

// The split of K over the grid for few rows: as split_rows (rows.cuh), with partial sums of at most
// half of W's bytes.
void split_bytes(ByteWork &w, long long slots) {
    w.across = (w.N + BYTE_COLS - 1) / BYTE_COLS;
    constexpr int step = BYTE_THREADS / 32 * 4 * BYTE_STEP;
    const long long steps = (w.K + step - 1LL) / step, fewest = (w.K + BYTE_RANGE - 1LL) / BYTE_RANGE;
    const long long most = std::max(fewest, std::min(steps, (long long)w.K / (16LL * w.M)));
    long long least = 0;
    for (long long n = fewest; n <= std::min(most, fewest + 64); ++n) {
        const long long per = (steps + n - 1) / n;
        const long long cost = ((w.across * n + slots - 1) / slots) * (per + 2);
        if (n == fewest || cost < least) least = cost, w.range = int(per * step);
    }
    w.ranges = int((w.K + (long long)w.range - 1) / w.range);
}

// The tiles of up to 256 rows and their ranges: the fewest us over the counts of ranges, with 0.19
// us for each slab of W that an SM reads, 2 to fill and empty a block, and the ranges' sums
// written and read once at 5 TB/s.
TileWork tiles_of(const Call &c, int sms) {
    TileWork w{};
    w.M = c.M, w.N = c.N, w.K = c.K;
    w.across = (c.N + TILE_COLS - 1) / TILE_COLS;
    w.down = (c.M + 255) / 256;
    w.rows = ((c.M + w.down - 1) / w.down + 15) / 16 * 16;
    w.timeout_ns = sgh::wait_timeout_ns();
    const int blocks = w.rows <= 64 ? 2 : 1, slabs = (c.K + TILE_K - 1) / TILE_K;
    const long long fewest = (c.K + TILE_RANGE - 1LL) / TILE_RANGE, slots = (long long)blocks * sms;
    double least = 0;
    for (long long n = fewest; n <= std::min<long long>(slabs, fewest + 64); ++n) {
        const long long per = (slabs + n - 1) / n;
        if ((slabs + per - 1) / per != n) continue;   // a range would be empty
        const long long items = (long long)w.across * w.down * n, waves = (items + slots - 1) / slots;
        const double cost = double(waves) * (double(per) * 0.19 * blocks + 2.0) + (n > 1 ? 2.0 + double(n) * c.M * c.N * 8.0 / 5.0e6 : 0.0);
        if (w.ranges == 0 || cost < least) least = cost, w.ranges = int(n), w.range = int(per * TILE_K);
    }
    return w;
}

template <class T, bool ALIGNED>
int launch_tiles(const Call &c, const TileWork &w) {
    const auto go = [&](auto of) {
        constexpr int ROWS = decltype(of)::value;
        using Z = ByteTile<ROWS, ALIGNED>;
        const auto kernel = byte_tiles_kernel<T, ROWS, ALIGNED>;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Z::SMEM));
        if (e != cudaSuccess) return sgh::cuda_fail(e);
        const long long blocks = (long long)w.across * w.down * w.ranges;
        if (blocks > 0x7fffffffLL) return int(SGEMM_ERR_TOO_LARGE);
        return sgh::launch("int8 as float16, tcgen05, W converted on its way", kernel, dim3(unsigned(blocks)), TILE_THREADS, Z::SMEM,
                           c.stream, w, c.q, c.ldq, c.W, (long long)c.ldw, c.scale, c.wscale, static_cast<const T *>(c.bias),
                           static_cast<T *>(c.Y), (long long)c.ldy);
    };
    return w.rows <= 32   ? go(std::integral_constant<int, 32>{})
           : w.rows <= 64 ? go(std::integral_constant<int, 64>{})
           : w.rows <= 128 ? go(std::integral_constant<int, 128>{})
                           : go(std::integral_constant<int, 256>{});
}

template <class T>
int finish(const Call &c, int ranges, const int *partial) {
    return sgh::launch(nullptr, byte_finish_kernel<T>, dim3(unsigned((c.N + 255LL) / 256), unsigned(std::min(c.M, 65535))), 256, 0,
                       c.stream, c.M, c.N, ranges, partial, c.scale, c.wscale, static_cast<const T *>(c.bias),
                       static_cast<T *>(c.Y), (long long)c.ldy);
}

int few_rows_most() { const char *e = getenv("L8_FEW"); return e ? atoi(e) : BYTE_ROWS; }
int tiles_most() { const char *e = getenv("L8_TILES"); return e ? atoi(e) : 512; }

template <class T>
int linear8(Call c) {
    int sms, st;
    cudaMemPool_t pool;
    if ((st = sgh::current_device(&sms, &pool)) != SGEMM_OK) return st;
    const bool own_rows = c.X != nullptr && c.K > 0, few = c.M <= few_rows_most(), tiles = !few && c.M <= tiles_most();
    const long long qpitch = (c.K + 15LL) / 16 * 16, xpitch = pitch8(c.K), wpitch = pitch8(c.N);
    const size_t q_bytes = own_rows ? size_t(c.M) * qpitch : 0, s_floats = own_rows ? c.M : 0;
    const bool pack = !few && !tiles;
    const size_t x_elems = pack ? size_t(c.M) * xpitch : 0, w_elems = pack ? size_t(c.K) * wpitch : 0;
    ByteWork w{};
    TileWork tw{};
    sgp::Split split{1, 256, 0};
    size_t p_ints = 0;
    if (c.K == 0) {
    } else if (few) {
        w.M = c.M, w.N = c.N, w.K = c.K;
        split_bytes(w, (c.M <= 4 ? 2LL : 1LL) * sms);
        p_ints = size_t(w.ranges) * c.M * c.N;
    } else if (tiles) {
        tw = tiles_of(c, sms);
        p_ints = tw.ranges > 1 ? size_t(tw.ranges) * c.M * c.N : 0;
    } else {
        split = sgq::plan(sgq::BYTES, c.M, c.N, c.K, 1, sms);
        p_ints = split.partial_floats;
    }
    sgh::Workspace ws(pool, c.stream);
    const auto piece = [](size_t n) { return sgh::Workspace::piece(n); };
    st = ws.allocate(piece(q_bytes) + piece(s_floats * 4) + piece(x_elems * 2) + piece(w_elems * 2) + piece(p_ints * 4));
    if (st != SGEMM_OK) return st;
    signed char *q = ws.take<signed char>(q_bytes);
    float *scale = ws.take<float>(s_floats);
    const Parts xp{ws.take<bf16>(x_elems), xpitch, c.M * xpitch}, wp{ws.take<bf16>(w_elems), wpitch, c.K * wpitch};
    int *partial = p_ints ? ws.take<int>(p_ints) : nullptr;
    if (own_rows) {
        if ((st = sgh::rows8(c.type, c.M, c.K, c.X, c.ldx, q, qpitch, scale, sms, c.stream)) != SGEMM_OK) return st;
        c.q = q, c.ldq = qpitch, c.scale = scale;
    }
    if (c.K == 0) {
        st = finish<T>(c, 0, nullptr);
    } else if (few) {
        w.partial = partial;
        const bool wide = sgh::aligned(c.W, 16) && c.ldw % 16 == 0;
        auto pick = [&](auto of) {
            constexpr bool V = decltype(of)::value;
            return c.M <= 1 ? byte_rows_kernel<1, V> : c.M <= 2 ? byte_rows_kernel<2, V> : c.M <= 4 ? byte_rows_kernel<4, V> : byte_rows_kernel<8, V>;
        };
        const long long blocks = (long long)w.across * w.ranges;
        if (blocks > 0x7fffffffLL) return SGEMM_ERR_TOO_LARGE;
        st = sgh::launch("int8, few rows, W read once", wide ? pick(std::true_type{}) : pick(std::false_type{}),
                         dim3(unsigned(blocks)), BYTE_THREADS, 0, c.stream, w, c.q, c.ldq, c.W, (long long)c.ldw);
        if (st == SGEMM_OK) st = finish<T>(c, w.ranges, partial);
    } else if (tiles) {
        tw.partial = partial;
        const bool in_place = sgh::aligned(c.W, 16) && c.ldw % 16 == 0 && sgh::aligned(c.q, 16) && c.ldq % 16 == 0;
        st = in_place ? launch_tiles<T, true>(c, tw) : launch_tiles<T, false>(c, tw);
        if (st == SGEMM_OK && partial) st = finish<T>(c, tw.ranges, partial);
    } else {
        const PartsJob<ByteRows> a(ByteRows{c.q, c.ldq}, c.M, c.K, sgh::aligned(c.q, 8) && c.ldq % 8 == 0, xp);
        const PartsJob<ByteRows> b(ByteRows{c.W, c.ldw}, c.K, c.N, sgh::aligned(c.W, 8) && c.ldw % 8 == 0, wp);
        const unsigned blocks = unsigned(std::min<long long>((a.octets() + b.octets() + 255) / 256, 32LL * sms));
        st = sgh::launch(nullptr, parts_kernel<1, 1, ByteRows, ByteRows>, dim3(blocks), 256, 0, c.stream, a, b, false);
        if (st != SGEMM_OK) return st;
        sgq::Product g{c.M, c.N, c.K, {xp.p, c.K, c.M, 1, xpitch, c.M * xpitch}, {{wp.p, c.N, c.K, 1, wpitch, c.K * wpitch}, {}}};
        const sgq::Output<T> out{static_cast<T *>(c.Y), nullptr, nullptr, c.ldy, 0, 0, 0, c.scale, c.wscale, static_cast<const T *>(c.bias)};
        st = sgq::run<T, sgq::BYTES>(g, out, split, reinterpret_cast<float *>(partial), sms, c.stream);
        if (st == SGEMM_OK && partial) st = finish<T>(c, split.splits, partial);
    }
    return st == SGEMM_OK ? ws.release() : st;
}

}  // namespace

cudaError_t sgh::linear8_error_word(unsigned *v, bool clear) { return sgv::unit_error_word(v, clear); }

SGEMM_API int sgemm_linear8(int type, int M, int N, int K, const void *X, int ldx, const signed char *q, int ldq,
                            const float *scale, const signed char *W, int ldw, const float *wscale, const void *bias, void *Y,
                            int ldy, sgemm_stream_t stream) {
    const int st = sgh::check_sizes(type, {M, N, K});
    if (st != SGEMM_OK) return st;
    if (K > kMostTerms) return SGEMM_ERR_TOO_LARGE;
    if (M == 0 || N == 0) return SGEMM_OK;
    const size_t size = sgh::element_bytes(type);
    if ((K > 0 && ((X ? sgh::bad_matrix(X, ldx, K, size) : sgh::bad_matrix(q, ldq, K, 1) || sgh::bad_vector(scale, 4)) ||
                   sgh::bad_matrix(W, ldw, N, 1) || sgh::bad_vector(wscale, 4))) ||
        !sgh::aligned(bias, size) || sgh::bad_matrix(Y, ldy, N, size))
        return SGEMM_ERR_INVALID_ARG;
    const Call c{type, M, N, K, X, ldx, q, ldq, scale, W, ldw, wscale, bias, Y, ldy, reinterpret_cast<cudaStream_t>(stream)};
    return type == SGEMM_BF16 ? linear8<bf16>(c) : linear8<float>(c);
}
