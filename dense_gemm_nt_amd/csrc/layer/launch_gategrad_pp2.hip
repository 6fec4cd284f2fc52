// launch_gated_pp2.hip's tile with the pre-activations' gradients.
#define GNT_GATE_GRAD
#include "launch_gated_pp2.hip"
