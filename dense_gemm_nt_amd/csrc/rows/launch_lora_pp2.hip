// The 256 x 256 ping-pong tile with low-rank adapters added (lora_add), the
// weight K-major, or with GNT_LORA_BNM MN-major (the input gradient).
#include "rows_launch.hpp"

#define GNT_EXT_KERNEL(name) name##_lora
#define GNT_EXT_ARGS LoraArgs
#define GNT_EXT_ACC(p, acc, r0, c0, split, lane) lora_add<IN, 1, low_parts<IN, OUT> == 2, low_parts<IN, OUT>>(p, acc, r0, c0, split, lane);
#include "../gemm_nt_pp2.hpp"

#ifndef GNT_LORA_BNM
#define GNT_LORA_BNM false
#define GNT_LORA_NAME kLora_pp2
#endif

namespace gnt {

template <int IN, int OUT>
static hipError_t launch_pp2(const LoraArgs &a, unsigned grid, hipStream_t s)
{
    hipLaunchKernelGGL((gemm_nt_pp2_lora<IN, OUT, false, GNT_LORA_BNM>), dim3(grid), dim3(512), 0, s, a);
    return hipGetLastError();
}

LoraTable GNT_LORA_NAME = GNT_ROWS_TABLE(launch_pp2);

}  // namespace gnt
