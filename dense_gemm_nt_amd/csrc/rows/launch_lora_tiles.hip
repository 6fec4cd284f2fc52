// Kernel-template tiles with low-rank adapters added (lora_add).
#include "rows_launch.hpp"

#define GNT_EXT_KERNEL(name) name##_lora
#define GNT_EXT_ARGS LoraArgs
#define GNT_EXT_ACC(p, acc, r0, c0, split, lane) lora_add<IN, (STAGES > 2 ? 8 : 2), (STAGES > 2), low_parts<IN, OUT>>(p, acc, r0, c0, split, lane);
#include "../gemm_nt_kernel.hpp"

namespace gnt {

#define GNT_LORA_TILE(NAME, BM, WM, WN, ST, ROT)                                                     \
    template <int IN, int OUT>                                                                       \
    static hipError_t launch_##NAME(const LoraArgs &a, unsigned grid, hipStream_t s)                 \
    {                                                                                                \
        hipLaunchKernelGGL((gemm_nt_kernel_lora<BM, 128, 64, WM, WN, ST, IN, OUT, false, ROT>),      \
                           dim3(grid), dim3(WM * WN * 64), 0, s, a);                                 \
        return hipGetLastError();                                                                    \
    }                                                                                                \
    LoraTable kLora_##NAME = GNT_ROWS_TABLE(launch_##NAME);

#ifndef GNT_LORA_TILES_B
GNT_LORA_TILE(128_s4, 128, 2, 4, 4, false)
GNT_LORA_TILE(128_s4_rot, 128, 2, 4, 4, true)
#else
GNT_LORA_TILE(128_s2, 128, 2, 4, 2, false)
GNT_LORA_TILE(32_rot, 32, 1, 4, 6, true)
#endif

}  // namespace gnt
