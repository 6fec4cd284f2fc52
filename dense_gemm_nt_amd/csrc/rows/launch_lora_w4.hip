// The four-wave 256 x 128 tile with low-rank adapters added (lora_add).
#include "rows_launch.hpp"

#define GNT_EXT_KERNEL(name) name##_lora
#define GNT_EXT_ARGS LoraArgs
#define GNT_EXT_ACC(p, acc, r0, c0, split, lane) lora_add<IN, 8, true, low_parts<IN, OUT>>(p, acc, r0, c0, split, lane);
#include "../gemm_nt_w4.hpp"

namespace gnt {

template <int IN, int OUT>
static hipError_t launch_w4(const LoraArgs &a, unsigned grid, hipStream_t s)
{
    hipLaunchKernelGGL((gemm_nt_w4_lora<IN, OUT, 128>), dim3(grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

LoraTable kLora_w4 = GNT_ROWS_TABLE(launch_w4);

}  // namespace gnt
