// The routed ping-pong tile with both operands MN-major (weight gradient).
#define GNT_ROUTED_AM true
#define GNT_ROUTED_BNM true
#define GNT_ROUTED_NAME kRouted_pp2_mm
#include "launch_routed_pp2.hip"
