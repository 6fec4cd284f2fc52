// rows_launch.hpp -- launch tables of the tiles with an addition, one
// translation unit each (launch_*.hip); indexed [in dtype][out dtype].
#pragma once

#include "rows_common.hpp"

namespace gnt {

typedef hipError_t (*lora_fn)(const LoraArgs &, unsigned grid, hipStream_t);
typedef hipError_t (*routed_fn)(const RoutedArgs &, unsigned grid, hipStream_t);
typedef lora_fn LoraTable[2][3];
typedef routed_fn RoutedTable[2][3];

// the tiles with the adapters added before anything leaves the accumulators
extern LoraTable kLora_128_s4, kLora_128_s4_rot, kLora_128_s2, kLora_32_rot, kLora_w4, kLora_pp2,
    kLora_pp2_km, kLora_tile_km;
// the tiles over rows sorted by expert (each block finds its tile's expert from the
// offsets, routed_lookup): both operands K-major (three
// tile heights), the weights MN-major (input gradient), both MN-major (weight
// gradient)
extern RoutedTable kRouted_32, kRouted_128, kRouted_pp2, kRouted_pp2_km, kRouted_pp2_mm;
// and on the 128 x 128 tile for MN-major weights (rows_tile.hpp)
extern RoutedTable kRouted_tile_km;

}  // namespace gnt

#define GNT_ROWS_TABLE(F) {{F<0, 0>, F<0, 1>, F<0, 2>}, {F<1, 0>, F<1, 1>, F<1, 2>}}
