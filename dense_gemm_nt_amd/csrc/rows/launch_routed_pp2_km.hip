// The routed ping-pong tile with the weights MN-major (input gradient).
#define GNT_ROUTED_AM false
#define GNT_ROUTED_BNM true
#define GNT_ROUTED_NAME kRouted_pp2_km
#include "launch_routed_pp2.hip"
