// gemm_nt_ext.hpp -- extension points of the tile kernels.  Not set by this
// library's own translation units: its kernels have the names and the argument
// block below and nothing added.  A translation unit of rows/ or layer/ that needs a tile
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
//   GNT_EXT_SUM(p, acc, r0, c0, lane)  changes the sum of K splits after its reduction in the kernel
//   GNT_EXT_MAP(p, tm, tn, split)  in place of the block map, K splits among it; false where
//                         the block has no tile; may move p.A and p.B
//   GNT_EXT_TILE(p, tm, tn)  the tile's number in the launch (its partials and counter)
//   GNT_EXT_STORE(p, acc, r0, c0, stage, lane)  in place of a whole sum's store (after a
//                         reduction in the kernel; partials of a second pass are stored as
//                         ever), through the wave's share of the idle LDS
//   GNT_EXT_AHEAD 1       a wave with one 32 x 32 block reads all of a slab's fragments before its
//                         first MFMA (gemm_nt_kernel.hpp): with one MFMA a k-step, reading one
//                         k-step ahead leaves most of each read's latency to be waited for
//   GNT_EXT_PAIRED 1      B's rows alternate in groups of eight between two arrays of
//                         GNT_EXT_COLS(p) rows each: row R of B is row 8 (R / 16) + R mod 8 of
//                         array (R / 8) mod 2, which GNT_EXT_B(p, w) and GNT_EXT_LDB(p, w)
//                         name.  Eight rows are what one wave-wide load of a K-major B
//                         brings (and two of an MN-major one, four each), so a wave loads
//                         from one of the arrays only, and what belongs together ends up in
//                         one lane's accumulators (registers 8 u + 0..3 and 8 u + 4..7).
// (Included by every tile header, so without an include guard of its own.)
#ifndef GNT_EXT_KERNEL
#define GNT_EXT_KERNEL(name) name
#define GNT_EXT_ARGS KernelArgs
#endif
#ifndef GNT_EXT_ACC
#define GNT_EXT_ACC(p, acc, r0, c0, split, lane)
#endif
#ifndef GNT_EXT_SUM
#define GNT_EXT_SUM(p, acc, r0, c0, lane)
#endif
#ifndef GNT_EXT_AHEAD
#define GNT_EXT_AHEAD 0
#endif
#ifndef GNT_EXT_TILE
#define GNT_EXT_TILE(p, tm, tn) ((tm) * p.tiles_n + (tn))
#endif
#ifndef GNT_EXT_PAIRED
#define GNT_EXT_PAIRED 0
#define GNT_EXT_COLS(p) 0
#define GNT_EXT_B(p, w) p.B
#define GNT_EXT_LDB(p, w) p.ldb
#endif
