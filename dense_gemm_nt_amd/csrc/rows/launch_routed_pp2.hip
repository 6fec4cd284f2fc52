// The 256 x 256 ping-pong tile over rows sorted by expert (routed_lookup), by operand
// layout.
#include "rows_launch.hpp"

#define GNT_EXT_KERNEL(name) name##_routed
#define GNT_EXT_ARGS RoutedArgs
#define GNT_EXT_LOOKUP(p, tm, tn) routed_lookup(p, tm, tn)
#include "../gemm_nt_pp2.hpp"

#ifndef GNT_ROUTED_NAME
#define GNT_ROUTED_AM false
#define GNT_ROUTED_BNM false
#define GNT_ROUTED_NAME kRouted_pp2
#endif

namespace gnt {

template <int IN, int OUT>
static hipError_t launch_pp2(const RoutedArgs &a, unsigned grid, hipStream_t s)
{
    hipLaunchKernelGGL((gemm_nt_pp2_routed<IN, OUT, GNT_ROUTED_AM, GNT_ROUTED_BNM, 0, true>), dim3(grid),
                       dim3(512), 0, s, a);
    return hipGetLastError();
}

RoutedTable GNT_ROUTED_NAME = GNT_ROWS_TABLE(launch_pp2);

}  // namespace gnt
