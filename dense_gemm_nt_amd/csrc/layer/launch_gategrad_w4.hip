// launch_gated_w4.hip's tile with the pre-activations' gradients.
#define GNT_GATE_GRAD
#include "launch_gated_w4.hip"
