// Kernel-template tiles of the gated block (paired_ext.hpp).
#include "layer_launch.hpp"
#include "paired_ext.hpp"
#include "../gemm_nt_kernel.hpp"

namespace gnt {

#define GNT_GATED_TILE(NAME, BM, WM, WN, ST, ROT)                                                    \
    template <int IN, int OUT>                                                                       \
    static hipError_t launch_##NAME(const PairedArgs &a, unsigned grid, hipStream_t s)               \
    {                                                                                                \
        hipLaunchKernelGGL((GNT_EXT_KERNEL(gemm_nt_kernel)<BM, 128, 64, WM, WN, ST, IN, OUT, false, ROT>), \
                           dim3(grid), dim3(WM * WN * 64), 0, s, a);                                 \
        return hipGetLastError();                                                                    \
    }                                                                                                \
    GNT_PAIRED_TYPE GNT_PAIRED(NAME) = GNT_PAIRED_TABLE(launch_##NAME);

#ifndef GNT_GATED_TILES_B
GNT_GATED_TILE(128_s4, 128, 2, 4, 4, false)
GNT_GATED_TILE(128_s4_rot, 128, 2, 4, 4, true)
#else
GNT_GATED_TILE(128_s2, 128, 2, 4, 2, false)
GNT_GATED_TILE(32_rot, 32, 1, 4, 6, true)
#ifndef GNT_GATE_GRAD
GNT_GATED_TILE(128_s2_rot, 128, 2, 4, 2, true)
#endif
#endif

}  // namespace gnt
