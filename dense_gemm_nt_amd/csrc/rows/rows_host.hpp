// rows_host.hpp -- argument checks and workspace carving of the row-indexed
// entry points (host code).
#pragma once

#include <stdint.h>

#include <cmath>

#include "gemm_rows.h"
#include "../gemm_nt_plan.hpp"

namespace gnt {

constexpr int64_t kMaxSize = (int64_t)INT32_MAX;
// A launch has fewer than 2^32 threads: blocks of at most 512, and 64 rows to
// 256 threads of the low-rank products.
constexpr int64_t kMaxBlocks = (int64_t)1 << 23;
constexpr int64_t kMaxRows = (int64_t)1 << 30;

inline bool is_16bit(int dt) { return dt == GEMM_BF16 || dt == GEMM_FP16; }
inline bool is_out(int dt) { return is_16bit(dt) || dt == GEMM_FP32; }
inline int64_t size_of(int dt) { return dt == GEMM_FP32 ? 4 : 2; }

// Consecutive 256-byte aligned pieces of a workspace, or (base null) their sizes.
struct Carver {
    uint8_t *base;
    int64_t used = 0;
    template <typename T>
    T *take(int64_t count)
    {
        const int64_t at = used;
        used += cdiv(count * (int64_t)sizeof(T), 256) * 256;
        return reinterpret_cast<T *>(base ? base + at : nullptr);
    }
};

inline gemm_status_t check_workspace(const void *ws, int64_t have, int64_t need)
{
    if (need == 0)
        return GEMM_OK;
    if (!ws || have < need)
        return GEMM_ERR_INVALID_ARG;
    return (uintptr_t)ws % 256 ? GEMM_ERR_MISALIGNED : GEMM_OK;
}

// A 16-bit operand of rows of `row` elements at a pitch of `ld`.
inline gemm_status_t check_operand(const void *p, int64_t row, int64_t ld)
{
    if (ld < row)
        return GEMM_ERR_INVALID_ARG;
    if (ld >= kMaxLeadingDim)
        return GEMM_ERR_UNSUPPORTED;
    if (!p)
        return GEMM_ERR_INVALID_ARG;
    return (uintptr_t)p % 16 || ld % 8 ? GEMM_ERR_MISALIGNED : GEMM_OK;
}

inline gemm_status_t check_output(const void *p, int64_t row, int64_t ld, int dt)
{
    if (ld < row)
        return GEMM_ERR_INVALID_ARG;
    if (ld >= kMaxSize)
        return GEMM_ERR_UNSUPPORTED;
    if (!p)
        return GEMM_ERR_INVALID_ARG;
    return (uintptr_t)p % size_of(dt) ? GEMM_ERR_MISALIGNED : GEMM_OK;
}

// The plan of a product whose B is MN-major (an input gradient's): the ping-pong tile, or
// (`tile`) the 128 x 128 one of rows_tile.hpp, with partials of at most `bound` bytes.
struct GradPlan {
    Plan plan;
    bool tile;
};
inline GradPlan plan_mn_major(int64_t M, int64_t N, int64_t K, int64_t bound)
{
    GradPlan g{make_plan(M, N, K, bound, CFG_PP2_256x256, -1, 0), false};
    // The ping-pong tiles from a quarter of the machine on (product and gradient
    // parts, 4096 deep: 777 x 2048, 32 tiles, 51 us against 42 on the smaller tile;
    // 1024 x 4096, 64 tiles, 62 against 58; 2048 x 4096, 128 tiles, 84 against 91).
    if (cdiv(M, 256) * cdiv(N, 256) >= kNumCUs / 4)
        return g;
    Plan &p = g.plan;
    g.tile = true;
    p = Plan{};
    p.tiles_m = (int)cdiv(M, 128);
    p.tiles_n = (int)cdiv(N, 128);
    p.k_tiles = (int)cdiv(K, 64);
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
    // K splits while all blocks, two to a compute unit, run at once; at least 8
    // slabs each
    int64_t splits = std::max<int64_t>(1, std::min<int64_t>(2 * kNumCUs / tiles, p.k_tiles / 8));
    while (splits > 1 && (tiles * splits * 128 * 128 * 4 > bound || tiles * 4 > GEMM_COUNTER_BYTES))
        --splits;
    p.kt_per_split = (int)cdiv(p.k_tiles, splits);
    p.splits = p.k_tiles ? (int)cdiv(p.k_tiles, p.kt_per_split) : 1;
    p.group_m = std::min(4, p.tiles_m);
    p.grid = tiles * p.splits;
    if (p.splits > 1) {
        p.inreduce = 1;
        p.ws_bytes = p.grid * 128 * 128 * 4;
    }
    return g;
}

inline gemm_status_t check_epilogue(const gemm_epilogue_t *epi)
{
    if (!epi)
        return GEMM_OK;
    if (epi->bias_along < GEMM_BIAS_NONE || epi->bias_along > GEMM_BIAS_M ||
        epi->activation < GEMM_ACT_NONE || epi->activation > GEMM_ACT_GELU)
        return GEMM_ERR_INVALID_ARG;
    if (epi->bias_along != GEMM_BIAS_NONE && (!epi->bias || (uintptr_t)epi->bias % 4))
        return GEMM_ERR_INVALID_ARG;
    return std::isfinite(epi->alpha) && std::isfinite(epi->beta) ? GEMM_OK : GEMM_ERR_UNSUPPORTED;
}

}  // namespace gnt
