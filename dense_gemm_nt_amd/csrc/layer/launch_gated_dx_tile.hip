// The gated block's input gradient on the 128 x 128 tile for MN-major weights (rows_tile.hpp) and
// the 64 x 64 one (tile64.hpp); their k-rows come from the two weights in turn.
#include "layer_launch.hpp"
#include "tile64.hpp"

namespace gnt {

template <>
struct TileHooks<PairedArgs> : PlanTile<PairedArgs> {
    static constexpr bool kPaired = true;
    template <int IN, int OUT, int FN, int FM>
    static __device__ __forceinline__ void add(PairedArgs &p, f32x16 (&acc)[FN][FM], int r0, int, int, int lane)
    {
        unscale<IN, false>(p, acc, r0, lane);
    }
    static __device__ __forceinline__ const uint16_t *b(const PairedArgs &p, int w) { return w ? p.B2 : p.B; }
    static __device__ __forceinline__ int ldb(const PairedArgs &p, int w) { return w ? p.ldb2 : p.ldb; }
    static __device__ __forceinline__ int cols(const PairedArgs &p) { return p.cols; }
};

template <int IN, int OUT>
static hipError_t launch_dx(const PairedArgs &a, unsigned grid, hipStream_t s)
{
    hipLaunchKernelGGL((rows_tile<IN, OUT, PairedArgs>), dim3(grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int IN, int OUT>
static hipError_t launch_dx_64(const PairedArgs &a, unsigned grid, hipStream_t s)
{
    hipLaunchKernelGGL((tile64<IN, OUT, PairedArgs>), dim3(grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

PairedTable kGatedDx_tile = GNT_LAYER_TABLE(launch_dx);
PairedTable kGatedDx_64 = GNT_LAYER_TABLE(launch_dx_64);

}  // namespace gnt
