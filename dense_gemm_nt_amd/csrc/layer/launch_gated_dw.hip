// The gated block's weight gradients on the ping-pong tile, both in one launch: the
// pre-activations' gradients and the input, both MN-major, the result's rows in turn groups
// of eight to the two weights.
#include "layer_launch.hpp"

#define GNT_EXT_KERNEL(name) name##_gated_dw
#define GNT_EXT_ARGS PairedArgs
#define GNT_EXT_ACC(p, acc, r0, c0, split, lane) unscale<IN, true>(p, acc, r0, lane);
#define GNT_EXT_STORE(p, acc, r0, c0, stage, lane) store_paired_rows<OUT>(p, acc, r0, c0, stage, lane)
#include "../gemm_nt_pp2.hpp"

namespace gnt {

template <int IN, int OUT>
static hipError_t launch_dw(const PairedArgs &a, unsigned grid, hipStream_t s)
{
    hipLaunchKernelGGL((gemm_nt_pp2_gated_dw<IN, OUT, true, true>), dim3(grid), dim3(512), 0, s, a);
    return hipGetLastError();
}

PairedTable kGatedDw_pp2 = GNT_LAYER_TABLE(launch_dw);

}  // namespace gnt
