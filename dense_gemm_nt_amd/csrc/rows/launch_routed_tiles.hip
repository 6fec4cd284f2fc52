// Kernel-template tiles over rows sorted by expert (routed_lookup).
#include "rows_launch.hpp"

#define GNT_EXT_KERNEL(name) name##_routed
#define GNT_EXT_ARGS RoutedArgs
#define GNT_EXT_LOOKUP(p, tm, tn) routed_lookup(p, tm, tn)
#include "../gemm_nt_kernel.hpp"

namespace gnt {

#define GNT_ROUTED_TILE(NAME, BM, WM, WN, ST)                                                        \
    template <int IN, int OUT>                                                                       \
    static hipError_t launch_##NAME(const RoutedArgs &a, unsigned grid, hipStream_t s)               \
    {                                                                                                \
        hipLaunchKernelGGL((gemm_nt_kernel_routed<BM, 128, 64, WM, WN, ST, IN, OUT, false, true>),   \
                           dim3(grid), dim3(WM * WN * 64), 0, s, a);                                 \
        return hipGetLastError();                                                                    \
    }                                                                                                \
    RoutedTable kRouted_##NAME = GNT_ROWS_TABLE(launch_##NAME);

GNT_ROUTED_TILE(32, 32, 1, 4, 6)
GNT_ROUTED_TILE(128, 128, 2, 4, 4)

}  // namespace gnt
