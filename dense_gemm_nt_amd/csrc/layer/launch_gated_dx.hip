// The gated block's input gradient on the ping-pong tile: the pre-activations'
// gradients, in turn groups of eight columns, by both weights MN-major.
#include "layer_launch.hpp"

#define GNT_EXT_KERNEL(name) name##_gated_dx
#define GNT_EXT_ARGS PairedArgs
#define GNT_EXT_PAIRED 1
#define GNT_EXT_COLS(p) (p.cols)
#define GNT_EXT_B(p, w) ((w) ? p.B2 : p.B)
#define GNT_EXT_LDB(p, w) ((w) ? p.ldb2 : p.ldb)
#define GNT_EXT_ACC(p, acc, r0, c0, split, lane) unscale<IN, false>(p, acc, r0, lane);
#include "../gemm_nt_pp2.hpp"

namespace gnt {

template <int IN, int OUT>
static hipError_t launch_dx(const PairedArgs &a, unsigned grid, hipStream_t s)
{
    hipLaunchKernelGGL((gemm_nt_pp2_gated_dx<IN, OUT, false, true>), dim3(grid), dim3(512), 0, s, a);
    return hipGetLastError();
}

PairedTable kGatedDx_pp2 = GNT_LAYER_TABLE(launch_dx);

}  // namespace gnt
