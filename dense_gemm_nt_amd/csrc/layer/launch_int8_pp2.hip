// The 256 x 256 ping-pong tile and the four-wave 256 x 128 one of the product in 8-bit
// integers.
#include "layer_launch.hpp"
#include "int8_ext.hpp"
#include "../gemm_nt_pp2.hpp"
#include "../gemm_nt_w4.hpp"

namespace gnt {

template <int OUT>
static hipError_t launch_pp2(const Int8Args &a, unsigned grid, hipStream_t s)
{
    hipLaunchKernelGGL((gemm_nt_pp2_int8<IN_I8, OUT>), dim3(grid), dim3(512), 0, s, a);
    return hipGetLastError();
}

template <int OUT>
static hipError_t launch_w4(const Int8Args &a, unsigned grid, hipStream_t s)
{
    hipLaunchKernelGGL((gemm_nt_w4_int8<IN_I8, OUT, 128>), dim3(grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

Int8Table kInt8_pp2 = {launch_pp2<0>, launch_pp2<1>, launch_pp2<2>};
Int8Table kInt8_w4 = {launch_w4<0>, launch_w4<1>, launch_w4<2>};

}  // namespace gnt
