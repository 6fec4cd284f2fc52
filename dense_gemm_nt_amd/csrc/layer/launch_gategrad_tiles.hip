// launch_gated_tiles.hip's tiles with the pre-activations' gradients.
#define GNT_GATE_GRAD
#include "launch_gated_tiles.hip"
