// rows_routed.hip -- host side of the experts' products over rows sorted by
// expert: argument checks, the tile by the rows per expert, one launch.
#include "rows_host.hpp"
#include "rows_launch.hpp"

namespace gnt {
namespace {

gemm_status_t check_sizes(int64_t rows, int64_t N, int64_t K, int64_t E, int in_dtype, int out_dtype)
{
    if (rows < 0 || N < 0 || K < 0 || E < 0)
        return GEMM_ERR_INVALID_ARG;
    if (!is_16bit(in_dtype) || !is_out(out_dtype))
        return GEMM_ERR_UNSUPPORTED;
    if (rows >= kMaxSize || N >= kMaxSize || K >= kMaxSize || E > 1024 || K % 8)
        return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

void fill_output(RoutedArgs &a, void *C, int64_t ldc, int out_dtype)
{
    const int64_t size = size_of(out_dtype);
    a.C = C;
    a.ldc = (int)ldc;
    a.c_size = (int)size;
    a.vec_store = ldc % 4 == 0 && (uintptr_t)C % (4 * size) == 0;
    a.rows16 = (ldc * size) % 16 == 0 && (uintptr_t)C % 16 == 0;
    a.group_m = 4;
    a.alpha = 1.0f;
}

// Tiles of `height` rows that the experts' rows make, as the host may expect it,
// who knows their number alone: rows of an expert spread evenly from none to twice
// the average, of which ceil(rows / height) has the mean below.
double expected_tiles(int64_t rows, int64_t E, int64_t height)
{
    const int64_t live = std::min(E, rows);
    const double r = 2.0 * (double)rows / (double)(std::max<int64_t>(1, live) * height);
    const double f = std::floor(r);
    return (double)live * (r <= 1.0 ? 1.0 : (f * (f + 1.0) / 2.0 + (r - f) * (f + 1.0)) / r);
}

// The height of K-major tiles: the least passes over the machine (a tile a
// compute unit), weighed by what a pass takes, 18 : 24 : 62 us for 32 x 128, 128 x
// 128 and 256 x 256 at a depth of 2048 (taken for every depth: their ratio is what
// counts).  (A pass a tenth over counts as not over.)
// Measured in us with 32 / 128 / 256 rows, depth 2048: 8 experts, N 2048: 320 rows
// 21 / 25 / 42, 512 rows 31 / 26 / 43, 2400 rows 76 / 47 / 57; 16 experts, N 4096: 640 rows
// 70 / 66 / 69, 1600 rows 116 / 84 / 73, 3200 rows 211 / 100 / 127, 7200 rows 415 / 202 / 166.
int tile_height(int64_t rows, int64_t N, int64_t E)
{
    int best = 0;
    double least = 0.0;
    for (int h : {32, 128, 256}) {
        const double tiles = expected_tiles(rows, E, h) * (double)cdiv(N, h == 256 ? 256 : 128);
        const double passes = std::max(1.0, std::ceil(tiles / kNumCUs - 0.1));
        const double cost = passes * (h == 32 ? 18.0 : h == 128 ? 24.0 : 62.0);
        if (best == 0 || cost < least)
            best = h, least = cost;
    }
    return best;
}

gemm_status_t launch(routed_fn fn, const RoutedArgs &a, int64_t tiles, hipStream_t stream)
{
    // whole runs of 256 blocks: the launch order permutes ids within them
    const int64_t grid = cdiv(tiles, 256) * 256;
    if (grid >= kMaxBlocks)
        return GEMM_ERR_UNSUPPORTED;
    return fn(a, (unsigned)grid, stream) == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

}  // namespace
}  // namespace gnt

using namespace gnt;

extern "C" {

gemm_status_t gemm_run_routed(const void *X, const void *W, void *C, const int32_t *offsets,
                              int64_t rows, int64_t N, int64_t K, int64_t num_experts, int64_t ldx,
                              int64_t ldw, int64_t w_stride, int64_t ldc, int layout_w,
                              int in_dtype, int out_dtype, int tail, hipStream_t stream)
{
    gemm_status_t st = check_sizes(rows, N, K, num_experts, in_dtype, out_dtype);
    if (st != GEMM_OK)
        return st;
    if ((layout_w != GEMM_K_MAJOR && layout_w != GEMM_MN_MAJOR) ||
        (tail != GEMM_TAIL_KEEP && tail != GEMM_TAIL_ZERO) || w_stride < 0)
        return GEMM_ERR_INVALID_ARG;
    if (rows == 0 || N == 0)
        return GEMM_OK;
    const bool mn = layout_w == GEMM_MN_MAJOR;
    if (!offsets || (st = check_output(C, N, ldc, out_dtype)) != GEMM_OK)
        return offsets ? st : GEMM_ERR_INVALID_ARG;
    if ((uintptr_t)offsets % 4)
        return GEMM_ERR_MISALIGNED;
    if (K > 0 && num_experts > 0) {
        if ((st = check_operand(X, K, ldx)) != GEMM_OK || (st = check_operand(W, mn ? N : K, ldw)) != GEMM_OK)
            return st;
        if (w_stride % 8)
            return GEMM_ERR_MISALIGNED;
    }
    RoutedArgs a{};
    a.A = static_cast<const uint16_t *>(X);
    a.B = static_cast<const uint16_t *>(W);
    a.lda = (int)ldx;
    a.ldb = (int)ldw;
    a.offsets = offsets;
    a.experts = (int)num_experts;
    a.rows = (int)rows;
    a.tail = tail == GEMM_TAIL_ZERO;
    a.b_stride = w_stride;
    a.N = (int)N;
    a.K = (int)K;
    fill_output(a, C, ldc, out_dtype);
    // sum of ceil(rows_e / height) over the experts and the tail, at most
    auto tall = [&](int64_t height) { return std::min<int64_t>(num_experts + 1, rows) + rows / height; };
    routed_fn fn;
    int bn = 256;
    a.tile_m = 256;
    if (mn && tall(256) * cdiv(N, 256) <= kNumCUs + cdiv(N, 256)) {
        // MN-major weights: the 128 x 128 tile while the ping-pong tiles would not
        // fill the machine once (8 experts, 2048 x 4096: 1024 rows 34 us against 55,
        // 2048 rows 55 against 61, 4096 rows 110 against 66)
        a.tile_m = bn = 128;
        fn = kRouted_tile_km[in_dtype][out_dtype];
    } else if (mn) {
        fn = kRouted_pp2_km[in_dtype][out_dtype];
    } else {
        a.tile_m = tile_height(rows, N, num_experts);
        bn = a.tile_m == 256 ? 256 : 128;
        fn = (a.tile_m == 256 ? kRouted_pp2 : a.tile_m == 128 ? kRouted_128 : kRouted_32)[in_dtype][out_dtype];
    }
    a.tiles_n = (int)cdiv(N, bn);
    // (and a tile row more where rows before the first expert's are a run of their own)
    return launch(fn, a, (tall(a.tile_m) + (a.tail ? 1 : 0)) * a.tiles_n, stream);
}

gemm_status_t gemm_run_routed_wgrad(const void *dY, const void *X, void *dW,
                                    const int32_t *offsets, int64_t rows, int64_t N, int64_t K,
                                    int64_t num_experts, int64_t lddy, int64_t ldx, int in_dtype,
                                    int out_dtype, hipStream_t stream)
{
    gemm_status_t st = check_sizes(rows, N, K, num_experts, in_dtype, out_dtype);
    if (st != GEMM_OK)
        return st;
    if (N % 8)
        return GEMM_ERR_UNSUPPORTED;
    if (N == 0 || K == 0 || num_experts == 0)
        return GEMM_OK;
    if (!offsets || (st = check_output(dW, K, K, out_dtype)) != GEMM_OK)
        return offsets ? st : GEMM_ERR_INVALID_ARG;
    if ((uintptr_t)offsets % 4)
        return GEMM_ERR_MISALIGNED;
    if (rows > 0 &&
        ((st = check_operand(dY, N, lddy)) != GEMM_OK || (st = check_operand(X, K, ldx)) != GEMM_OK))
        return st;
    RoutedArgs a{};
    a.A = static_cast<const uint16_t *>(dY);
    a.B = static_cast<const uint16_t *>(X);
    a.lda = (int)lddy;
    a.ldb = (int)ldx;
    a.offsets = offsets;
    a.experts = (int)num_experts;
    a.rows = (int)rows;
    a.wgrad = 1;
    a.tile_m = 256;
    a.c_stride = N * K;
    a.M = (int)N;
    a.N = (int)K;
    fill_output(a, dW, K, out_dtype);
    // (each expert's array starts N K elements after the last one's: of 8 values)
    // One expert's tiles after the other's, so that their panels meet in the L2s.  16384
    // rows of 32 uneven experts, 2048 x 4096, FP32 results 449 us, of which the
    // stores alone (no rows) take 179.  Experts' tiles taking turns, so that one's
    // stores would run under another's products, was slower: 2, 4 and 8 at a time by 4, 13
    // and 18%.
    a.tiles_n = (int)cdiv(K, 256);
    return launch(kRouted_pp2_mm[in_dtype][out_dtype], a, num_experts * cdiv(N, 256) * a.tiles_n, stream);
}

}  // extern "C"
