// ortho_ext.hpp -- the tiles' extension points for the orthogonalized update (before a tile
// header).
#define GNT_EXT_KERNEL(name) name##_ortho
#define GNT_EXT_AHEAD 1
#define GNT_EXT_ARGS OrthoArgs
#define GNT_EXT_MAP(p, tm, tn, split) ortho_map(p, tm, tn, split)
#define GNT_EXT_TILE(p, tm, tn) ortho_tile(p)
#define GNT_EXT_STORE(p, acc, r0, c0, stage, lane) store_ortho(p, acc, r0, c0, stage, lane)
