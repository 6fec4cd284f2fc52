// rows_index.hpp -- index arithmetic of the row-indexed kernels that the host can
// check, too (plain C++).
#pragma once

#include <stdint.h>

#ifdef __HIP__
#define GNT_BOTH __host__ __device__
#else
#define GNT_BOTH
#endif

namespace gnt {

// The words that a thread of a grid of blocks clears: first, first + step, ... below a
// count.  In 64 bits: the low-rank product of 2^30 rows has 2^24 blocks a K split, whose
// threads' numbers pass 2^31 (a negative one would be below every count).
struct Walk {
    int64_t first, step;
};

GNT_BOTH constexpr Walk clear_walk(uint32_t x, uint32_t y, uint32_t z, uint32_t grid_x, uint32_t grid_y, uint32_t grid_z,
                                   uint32_t threads, uint32_t thread)
{
    return Walk{(((int64_t)z * grid_y + y) * grid_x + x) * threads + thread,
                (int64_t)grid_x * grid_y * grid_z * threads};
}

}  // namespace gnt
