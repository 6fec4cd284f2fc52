// launch_gated_tiles_b.hip's tiles with the pre-activations' gradients.
#define GNT_GATE_GRAD
#define GNT_GATED_TILES_B
#include "launch_gated_tiles.hip"
