// The 256 x 256 ping-pong tile of the gated block (paired_ext.hpp).
#include "layer_launch.hpp"
#include "paired_ext.hpp"
#include "../gemm_nt_pp2.hpp"

namespace gnt {

template <int IN, int OUT>
static hipError_t launch_pp2(const PairedArgs &a, unsigned grid, hipStream_t s)
{
    hipLaunchKernelGGL((GNT_EXT_KERNEL(gemm_nt_pp2)<IN, OUT>), dim3(grid), dim3(512), 0, s, a);
    return hipGetLastError();
}

GNT_PAIRED_TYPE GNT_PAIRED(pp2) = GNT_PAIRED_TABLE(launch_pp2);

}  // namespace gnt
