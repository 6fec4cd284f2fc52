// paired_ext.hpp -- the tiles' extension points for B in two arrays (before a tile header):
// the gated block, or with GNT_GATE_GRAD its pre-activations' gradients.
#define GNT_EXT_AHEAD 1
#define GNT_EXT_ARGS PairedArgs
#define GNT_EXT_PAIRED 1
#define GNT_EXT_COLS(p) (p.cols)
#define GNT_EXT_B(p, w) ((w) ? p.B2 : p.B)
#define GNT_EXT_LDB(p, w) ((w) ? p.ldb2 : p.ldb)
#ifdef GNT_GATE_GRAD
#define GNT_EXT_KERNEL(name) name##_gategrad
#define GNT_EXT_STORE(p, acc, r0, c0, stage, lane) store_gate_gradients<IN>(p, acc, r0, c0, stage, lane)
#define GNT_PAIRED(name) kGateGrad_##name
#define GNT_PAIRED_TABLE(F) {F<0, 0>, F<1, 1>}
#define GNT_PAIRED_TYPE PairedInTable
#else
#define GNT_EXT_KERNEL(name) name##_gated
#define GNT_EXT_STORE(p, acc, r0, c0, stage, lane) store_gated<OUT>(p, acc, r0, c0, stage, lane)
#define GNT_PAIRED(name) kGated_##name
#define GNT_PAIRED_TABLE(F) GNT_LAYER_TABLE(F)
#define GNT_PAIRED_TYPE PairedTable
#endif
