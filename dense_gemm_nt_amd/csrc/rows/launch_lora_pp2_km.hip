// The ping-pong tile with low-rank adapters added, the weight MN-major.
#define GNT_LORA_BNM true
#define GNT_LORA_NAME kLora_pp2_km
#include "launch_lora_pp2.hip"
