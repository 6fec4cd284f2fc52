// Kernel-template tiles with low-rank adapters added, part two.
#define GNT_LORA_TILES_B
#include "launch_lora_tiles.hip"
