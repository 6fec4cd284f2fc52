// gemm_nt_ext.hpp -- extension points of the tile kernels.  Not set by this
// library's own translation units: its kernels have the names and the argument
// block below and nothing added.  A translation unit of rows/ that needs a tile
// with an addition defines them before it includes a tile header:
//   GNT_EXT_KERNEL(name)  the kernel's name (its own, so that the two libraries'
//                         kernels stay apart)
//   GNT_EXT_ARGS          its argument block, derived from KernelArgs
//   GNT_EXT_LOOKUP(p, tm, tn)  in place of the block map: sets p's problem
//                         fields and the tile from the block id; false where the
//                         block has no tile (the ping-pong kernel with GR, and
//                         the kernel-template tiles, whose splits are then 1)
//   GNT_EXT_ACC(p, acc, r0, c0, split, lane)  adds to a wave's accumulators,
//                         whose block starts at row r0 and column c0, once the
//                         main loop is done and before anything leaves them
// (Included by every tile header, so without an include guard of its own.)
#ifndef GNT_EXT_KERNEL
#define GNT_EXT_KERNEL(name) name
#define GNT_EXT_ARGS KernelArgs
#endif
#ifndef GNT_EXT_ACC
#define GNT_EXT_ACC(p, acc, r0, c0, split, lane)
#endif
