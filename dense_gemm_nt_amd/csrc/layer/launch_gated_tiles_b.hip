// The other half of launch_gated_tiles.hip's tiles.
#define GNT_GATED_TILES_B
#include "launch_gated_tiles.hip"
