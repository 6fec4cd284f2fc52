// The tiles of the orthogonalized update: both operands K-major on three tile sizes, and the
// second MN-major (the step) on the ping-pong tile and the 128 x 128 one of rows_tile.hpp.
#include "layer_launch.hpp"
#include "ortho_common.hpp"
#include "ortho_ext.hpp"
#include "../gemm_nt_kernel.hpp"
#include "../gemm_nt_pp2.hpp"
#include "../rows/rows_tile.hpp"
#include "tile64.hpp"

namespace gnt {

template <>
struct TileHooks<OrthoArgs> : PlanTile<OrthoArgs> {
    static constexpr bool kStore = true;
    template <int IN, int OUT, int FN, int FM>
    static __device__ __forceinline__ void add(OrthoArgs &, f32x16 (&)[FN][FM], int, int, int, int)
    {
    }
    static __device__ __forceinline__ bool map(OrthoArgs &p, int &tm, int &tn, int &split)
    {
        return ortho_map(p, tm, tn, split);
    }
    static __device__ __forceinline__ int tile(const OrthoArgs &p, int, int) { return ortho_tile(p); }
    template <int FN, int FM>
    static __device__ __forceinline__ void store(const OrthoArgs &p, const f32x16 (&acc)[FN][FM], int r0, int c0,
                                                 uint8_t *stage, int lane)
    {
        store_ortho(p, acc, r0, c0, stage, lane);
    }
};

hipError_t launch_ortho(const OrthoArgs &a, OrthoTile tile, unsigned grid, hipStream_t s)
{
    switch (tile) {
    case ORTHO_256_MN:
        hipLaunchKernelGGL((gemm_nt_pp2_ortho<IN_FP16, OUT_FP16, false, true>), dim3(grid), dim3(512), 0, s, a);
        break;
    case ORTHO_256:
        hipLaunchKernelGGL((gemm_nt_pp2_ortho<IN_FP16, OUT_FP16>), dim3(grid), dim3(512), 0, s, a);
        break;
    case ORTHO_128_MN:
        hipLaunchKernelGGL((rows_tile<IN_FP16, OUT_FP16, OrthoArgs>), dim3(grid), dim3(256), 0, s, a);
        break;
    case ORTHO_128:
        hipLaunchKernelGGL((gemm_nt_kernel_ortho<128, 128, 64, 2, 4, 4, IN_FP16, OUT_FP16, false, false>), dim3(grid),
                           dim3(512), 0, s, a);
        break;
    case ORTHO_128_S2:
        hipLaunchKernelGGL((gemm_nt_kernel_ortho<128, 128, 64, 2, 4, 2, IN_FP16, OUT_FP16, false, false>), dim3(grid),
                           dim3(512), 0, s, a);
        break;
    case ORTHO_64:
        hipLaunchKernelGGL((gemm_nt_kernel_ortho<64, 64, 64, 2, 2, 4, IN_FP16, OUT_FP16, false, false>), dim3(grid),
                           dim3(256), 0, s, a);
        break;
    case ORTHO_64_MN:
        hipLaunchKernelGGL((tile64<IN_FP16, OUT_FP16, OrthoArgs>), dim3(grid), dim3(256), 0, s, a);
        break;
    }
    return hipGetLastError();
}

}  // namespace gnt
