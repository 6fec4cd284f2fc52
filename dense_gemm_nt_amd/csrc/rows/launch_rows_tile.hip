// The 128 x 128 tile for MN-major B (rows_tile.hpp): with adapters added, and
// over rows sorted by expert.
#include "rows_launch.hpp"
#include "rows_tile.hpp"

namespace gnt {

template <int IN, int OUT>
static hipError_t launch_lora(const LoraArgs &a, unsigned grid, hipStream_t s)
{
    hipLaunchKernelGGL((rows_tile<IN, OUT, LoraArgs>), dim3(grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int IN, int OUT>
static hipError_t launch_km(const RoutedArgs &a, unsigned grid, hipStream_t s)
{
    hipLaunchKernelGGL((rows_tile<IN, OUT, RoutedArgs>), dim3(grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

LoraTable kLora_tile_km = GNT_ROWS_TABLE(launch_lora);
RoutedTable kRouted_tile_km = GNT_ROWS_TABLE(launch_km);

}  // namespace gnt
