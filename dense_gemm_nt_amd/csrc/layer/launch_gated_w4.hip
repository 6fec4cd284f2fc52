// The four-wave 256 x 128 tile of the gated block (paired_ext.hpp).
#include "layer_launch.hpp"
#include "paired_ext.hpp"
#include "../gemm_nt_w4.hpp"

namespace gnt {

template <int IN, int OUT>
static hipError_t launch_w4(const PairedArgs &a, unsigned grid, hipStream_t s)
{
    hipLaunchKernelGGL((GNT_EXT_KERNEL(gemm_nt_w4)<IN, OUT, 128>), dim3(grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

GNT_PAIRED_TYPE GNT_PAIRED(w4) = GNT_PAIRED_TABLE(launch_w4);

}  // namespace gnt
