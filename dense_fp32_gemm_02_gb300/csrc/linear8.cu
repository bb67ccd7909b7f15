// linear8.cu -- entry point of the product of int8 matrices with scales for each row and column.
#include "layer_host.h"
#include "byte_rows.cuh"
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
    long long ldw;
    const float *wscale;
    const void *bias;
    void *Y;
    int ldy;
    cudaStream_t stream;
};

// The tiles of up to 256 rows and their ranges: the fewest us over the counts of ranges, with so
// many for each 128 k of a block, by its rows, and 5.5 to fill and empty it.
TileWork tiles_of(const Call &c, int sms) {
    TileWork w{};
    w.M = c.M, w.N = c.N, w.K = c.K;
    w.across = (c.N + TILE_COLS - 1) / TILE_COLS;
    w.down = (c.M + 255) / 256;
    w.rows = ((c.M + w.down - 1) / w.down + 15) / 16 * 16;
    w.timeout_ns = sgh::wait_timeout_ns();
    const int steps = (c.K + 127) / 128;
    const double slab = w.rows <= 32 ? 0.45 : w.rows <= 64 ? 0.6 : w.rows <= 128 ? 0.85 : 1.75;
    double least = 0;
    for (int n = 1; n <= std::min(steps, MOST_CLUSTER); ++n) {
        const int per = (steps + n - 1) / n;
        if ((steps + per - 1) / per != n) continue;   // a range would be empty
        const long long items = (long long)w.across * w.down * n, waves = (items + sms - 1) / sms;
        const double of = double(waves) * (per * slab + 5.5) + 0.25 * n;
        if (w.ranges == 0 || of < least) least = of, w.ranges = n, w.range = per * 128;
    }
    return w;
}

// Up to so many rows W is brought to float16 on its way (byte_tiles.cuh); more rows make it worth while to
// lay both matrices out as bfloat16 first.  us at 4096 x 4096, on its way / laid out: 64 rows 10.6 / 27.6,
// 256 rows 19.9 / 34.2, 512 rows 32 / 37, 1024 rows 57 / 38; 753 x 678 x 4443 36.8 / 22.
constexpr int kTileRows = 512;

int encode_bytes(CUtensorMap *map, const signed char *p, long long inner, long long outer, long long pitch, uint32_t box_inner,
                 uint32_t box_outer) {
    const cuuint64_t dims[2] = {cuuint64_t(inner), cuuint64_t(outer)}, strides[1] = {cuuint64_t(pitch)};
    const cuuint32_t box[2] = {box_inner, box_outer}, steps[2] = {1, 1};
    const CUresult r = sgh::encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<signed char *>(p), dims, strides, box,
                                           steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SGEMM_OK : sgh::driver_fail(int(r));
}

template <class T>
int launch_tiles(const Call &c, const TileWork &w) {
    const auto go = [&](auto of) {
        constexpr int ROWS = decltype(of)::value;
        using Z = ByteTile<ROWS>;
        const auto kernel = byte_tiles_kernel<T, ROWS>;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Z::SMEM));
        if (e != cudaSuccess) return sgh::cuda_fail(e);
        CUtensorMap mX, mW;
        int st = encode_bytes(&mX, c.q, c.K, c.M, c.ldq, Z::STEP, ROWS);
        if (st == SGEMM_OK) st = encode_bytes(&mW, c.W, c.N, c.K, c.ldw, TILE_COLS, Z::STEP);
        if (st != SGEMM_OK) return st;
        const long long blocks = (long long)w.across * w.down * w.ranges;
        if (blocks > 0x7fffffffLL) return int(SGEMM_ERR_TOO_LARGE);
        return sgh::launch_cluster("int8 as float16, tcgen05, W converted on its way", kernel, dim3(unsigned(blocks)), TILE_THREADS,
                                   Z::SMEM, w.ranges, c.stream, mX, mW, w, c.scale, c.wscale,
                                   static_cast<const T *>(c.bias), static_cast<T *>(c.Y), (long long)c.ldy);
    };
    return w.rows <= 32    ? go(std::integral_constant<int, 32>{})
           : w.rows <= 64  ? go(std::integral_constant<int, 64>{})
           : w.rows <= 128 ? go(std::integral_constant<int, 128>{})
                           : go(std::integral_constant<int, 256>{});
}

// Bytes whose rows are not 16-byte aligned, at a pitch where they are.
int pitched(const signed char *p, long long ld, int rows, int cols, signed char *out, long long pitch, int sms, cudaStream_t stream) {
    const Divisor per_row = Divisor::of(unsigned((cols + 15LL) / 16));
    const long long units = (long long)rows * per_row.d;
    return sgh::launch(nullptr, byte_pitch_kernel, dim3(unsigned(std::min<long long>((units + 255) / 256, 32LL * sms))), 256, 0, stream,
                       p, ld, rows, cols, per_row, out, pitch);
}

template <class T>
int finish(const Call &c, int ranges, const int *partial) {
    return sgh::launch(nullptr, byte_finish_kernel<T>, dim3(unsigned((c.N + 511LL) / 512), unsigned(std::min(c.M, 65535))), 128, 0,
                       c.stream, c.M, c.N, ranges, partial, c.scale, c.wscale, static_cast<const T *>(c.bias),
                       static_cast<T *>(c.Y), (long long)c.ldy);
}

bool aligned_rows(const signed char *p, long long ld, int to = 16) { return sgh::aligned(p, size_t(to)) && ld % to == 0; }

// One to four rows, unless their range of q in shared memory would be too long (byte_rows.cuh).  us so / by
// tiles, rows of bfloat16: at 4096 x 4096 one row 7.1 / 12.4, two 7.9 / 12.5, four 9.1 / 12.6; four at 8192 x 8192
// 23 / 25, at 65536 x 1024 72 / 45, at 8191 x 8191 35 / 46.
constexpr int kStreamedRows = 4;
bool streamed(const Call &c) {
    return c.M <= kStreamedRows && c.K > 0 && (long long)c.M * c.K <= MOST_CLUSTER * ROWS_RANGE;
}

// The ranges: the least of waves of two blocks to an SM times the steps of a block, with 3 to begin and end it.
template <class T, int ROWS, int TILE>
int stream(const Call &c, int sms) {
    constexpr int STEP = rows_step(TILE);
    const int across = (c.N + TILE - 1) / TILE, steps = (c.K + STEP - 1) / STEP;
    ByteRows<T> a{c.M, c.N, c.K, 0, 0, static_cast<const T *>(c.X), c.q, c.W, c.scale, c.wscale, static_cast<const T *>(c.bias),
                  static_cast<T *>(c.Y), c.ldx, c.ldq, c.ldw, c.ldy};
    long long least = 0;
    for (int n = 1; n <= std::min(steps, MOST_CLUSTER); ++n) {
        const int per = (steps + n - 1) / n;
        if ((steps + per - 1) / per != n || per * STEP > ROWS_RANGE) continue;   // a range would be empty, or too long
        const long long cost = ((long long)across * n + 2 * sms - 1) / (2 * sms) * (per + 3);
        if (a.ranges == 0 || cost < least) least = cost, a.ranges = n, a.range = per * STEP;
    }
    const auto kernel = aligned_rows(c.W, c.ldw, ROWS == 4 ? 4 : 8) ? byte_rows_kernel<T, ROWS, TILE, true> : byte_rows_kernel<T, ROWS, TILE, false>;
    const size_t smem = byte_rows_smem<ROWS, TILE>(a.range);
    // Over the 48 KB that need no leave, with what the kernel declares itself.  The leave is for the most that any call
    // takes: threads share it, and a call's own size would take another thread's launch its leave away.
    if (smem > 40960) {
        constexpr size_t most = byte_rows_smem<ROWS, TILE>(ROWS_RANGE);
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(most));
        if (e != cudaSuccess) return sgh::cuda_fail(e);
    }
    return sgh::launch_cluster("int8, W streamed to few rows", kernel, dim3(unsigned(across * a.ranges)), ROWS_THREADS, smem, a.ranges,
                               c.stream, a);
}

template <class T>
int linear8(Call c) {
    int sms, st;
    cudaMemPool_t pool;
    if ((st = sgh::current_device(&sms, &pool)) != SGEMM_OK) return st;
    if (streamed(c)) {
        // (columns whose tiles of 128 would leave SMs without a block; 16384 x 1024, tiles of 64 / 128: 7.2 / 10.5 us)
        const bool narrow = (long long)(c.N + 127) / 128 * MOST_CLUSTER <= sms;
        return c.M > 2    ? stream<T, 4, 128>(c, sms)
               : c.M == 2 ? stream<T, 2, 128>(c, sms)
               : narrow   ? stream<T, 1, 64>(c, sms)
                          : stream<T, 1, 128>(c, sms);
    }
    const bool own_rows = c.X != nullptr && c.K > 0, tiles = c.M <= kTileRows;
    const long long qpitch = (c.K + 15LL) / 16 * 16, xpitch = pitch8(c.K), wpitch = pitch8(c.N), bpitch = (c.N + 15LL) / 16 * 16;
    const size_t q_bytes = own_rows ? size_t(c.M) * qpitch : 0, s_floats = own_rows ? c.M : 0;
    const size_t x_elems = tiles ? 0 : size_t(c.M) * xpitch, w_elems = tiles ? 0 : size_t(c.K) * wpitch;
    TileWork tw{};
    sgp::Split split{1, 256, 0};
    size_t p_ints = 0, q_copy = 0, w_copy = 0;
    if (c.K == 0) {
    } else if (tiles) {
        tw = tiles_of(c, sms);
        if (!own_rows && !aligned_rows(c.q, c.ldq)) q_copy = size_t(c.M) * qpitch;
        if (!aligned_rows(c.W, c.ldw)) w_copy = size_t(c.K) * bpitch;
    } else {
        split = sgq::plan(sgq::BYTES, c.M, c.N, c.K, 1, sms);
        p_ints = split.partial_floats;
    }
    sgh::Workspace ws(pool, c.stream);
    const auto piece = [](size_t n) { return sgh::Workspace::piece(n); };
    st = ws.allocate(piece(q_bytes) + piece(s_floats * 4) + piece(x_elems * 2) + piece(w_elems * 2) + piece(p_ints * 4) +
                     piece(q_copy) + piece(w_copy) + piece(sizeof(int)));
    if (st != SGEMM_OK) return st;
    signed char *q = ws.take<signed char>(q_bytes);
    float *scale = ws.take<float>(s_floats);
    const Parts xp{ws.take<bf16>(x_elems), xpitch, c.M * xpitch}, wp{ws.take<bf16>(w_elems), wpitch, c.K * wpitch};
    int *partial = p_ints ? ws.take<int>(p_ints) : nullptr, *large = ws.take<int>(1);
    if (own_rows) {
        if ((st = sgh::rows8(c.type, c.M, c.K, c.X, c.ldx, q, qpitch, scale, sms, c.stream)) != SGEMM_OK) return st;
        c.q = q, c.ldq = qpitch, c.scale = scale;
    }
    if (c.K == 0) {
        st = finish<T>(c, 0, nullptr);
    } else if (tiles) {
        if (q_copy) {
            signed char *to = ws.take<signed char>(q_copy);
            if ((st = pitched(c.q, c.ldq, c.M, c.K, to, qpitch, sms, c.stream)) != SGEMM_OK) return st;
            c.q = to, c.ldq = qpitch;
        }
        if (w_copy) {
            signed char *to = ws.take<signed char>(w_copy);
            if ((st = pitched(c.W, c.ldw, c.K, c.N, to, bpitch, sms, c.stream)) != SGEMM_OK) return st;
            c.W = to, c.ldw = bpitch;
        }
        st = launch_tiles<T>(c, tw);
    } else {
        const auto expand = [&](auto kernel, const ByteJob &job) {
            const unsigned blocks = unsigned(std::min<long long>((job.items() + 7) / 8, 32LL * sms));
            return sgh::launch(nullptr, kernel, dim3(blocks), 256, 0, c.stream, job, large);
        };
        st = expand(byte_expand_kernel<false>, ByteJob{c.W, c.ldw, c.K, c.N, wp, aligned_rows(c.W, c.ldw, 8)});
        if (st == SGEMM_OK) st = expand(byte_expand_kernel<true>, ByteJob{c.q, c.ldq, c.M, c.K, xp, aligned_rows(c.q, c.ldq, 8)});
        if (st != SGEMM_OK) return st;
        sgq::Product g{c.M, c.N, c.K, {xp.p, c.K, c.M, 1, xpitch, c.M * xpitch}, {{wp.p, c.N, c.K, 1, wpitch, c.K * wpitch}, {}}};
        const sgq::Output<T> out{static_cast<T *>(c.Y), nullptr, nullptr, c.ldy, 0, 0, 0, c.scale, c.wscale, static_cast<const T *>(c.bias),
                                 partial ? nullptr : large};   // (with one range chunks begin at multiples of 2048)
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
