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
