// layer_launch.hpp -- launch tables of the tiles of a feed-forward layer's products, one
// translation unit each (launch_*.hip).
#pragma once

#include "layer_common.hpp"

namespace gnt {

typedef hipError_t (*paired_fn)(const PairedArgs &, unsigned grid, hipStream_t);
typedef hipError_t (*int8_fn)(const Int8Args &, unsigned grid, hipStream_t);
typedef paired_fn PairedTable[2][3];       // [in dtype][out dtype]
typedef paired_fn PairedInTable[2];        // [in dtype]
typedef int8_fn Int8Table[3];              // [out dtype]

// the gated block: act(gate) * up of the tile's sums
extern PairedTable kGated_128_s4, kGated_128_s4_rot, kGated_128_s2, kGated_128_s2_rot, kGated_32_rot, kGated_w4, kGated_pp2;
// its pre-activations' gradients from the same sums
extern PairedInTable kGateGrad_128_s4, kGateGrad_128_s4_rot, kGateGrad_128_s2, kGateGrad_32_rot, kGateGrad_w4,
    kGateGrad_pp2;
// the gradients in the input (the weights MN-major) and in the weights (both operands
// MN-major)
extern PairedTable kGatedDx_pp2, kGatedDx_tile, kGatedDx_64, kGatedDw_pp2;
// the product in 8-bit integers
extern Int8Table kInt8_128_s4, kInt8_128_s4_rot, kInt8_128_s2, kInt8_128_s2_rot, kInt8_32_rot, kInt8_w4, kInt8_pp2;

}  // namespace gnt

#define GNT_LAYER_TABLE(F) {{F<0, 0>, F<0, 1>, F<0, 2>}, {F<1, 0>, F<1, 1>, F<1, 2>}}
