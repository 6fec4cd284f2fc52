// Kernel-template tiles of the product in 8-bit integers.
#include "layer_launch.hpp"
#include "int8_ext.hpp"
#include "../gemm_nt_kernel.hpp"

namespace gnt {

#define GNT_INT8_TILE(NAME, BM, WM, WN, ST, ROT)                                                     \
    template <int OUT>                                                                               \
    static hipError_t launch_##NAME(const Int8Args &a, unsigned grid, hipStream_t s)                 \
    {                                                                                                \
        hipLaunchKernelGGL((gemm_nt_kernel_int8<BM, 128, 64, WM, WN, ST, IN_I8, OUT, false, ROT>),   \
                           dim3(grid), dim3(WM * WN * 64), 0, s, a);                                 \
        return hipGetLastError();                                                                    \
    }                                                                                                \
    Int8Table kInt8_##NAME = {launch_##NAME<0>, launch_##NAME<1>, launch_##NAME<2>};

GNT_INT8_TILE(128_s4, 128, 2, 4, 4, false)
GNT_INT8_TILE(128_s4_rot, 128, 2, 4, 4, true)
GNT_INT8_TILE(128_s2, 128, 2, 4, 2, false)
GNT_INT8_TILE(128_s2_rot, 128, 2, 4, 2, true)
GNT_INT8_TILE(32_rot, 32, 1, 4, 6, true)

}  // namespace gnt
