// int8_ext.hpp -- the tiles' extension points for 8-bit integers (before a tile header).
#define GNT_EXT_KERNEL(name) name##_int8
#define GNT_EXT_AHEAD 1
#define GNT_EXT_ARGS Int8Args
// a whole sum's scales: of one split before the store, of several once they are added up
#define GNT_EXT_ACC(p, acc, r0, c0, split, lane) int8_scale(p, acc, r0, c0, lane, p.splits == 1);
#define GNT_EXT_SUM(p, acc, r0, c0, lane) int8_scale(p, acc, r0, c0, lane, true);
