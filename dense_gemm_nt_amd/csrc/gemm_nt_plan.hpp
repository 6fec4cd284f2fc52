// gemm_nt_plan.hpp -- the per-shape plan: which tile of the family a problem
// runs on, how its K is split, and the grid.  Host code only, shared by the
// libraries that launch these tiles (each with its own launch tables, indexed
// by CFG_*).
#pragma once

#include <stdint.h>
#include <string.h>

#include <algorithm>

// Per-tile arrival counters of the in-kernel two-split reduction, at the end of
// every workspace (handle or scratch): zero between calls (each call's second
// arrival resets its tile's counter).
#define GEMM_COUNTER_BYTES ((int64_t)64 << 10)

namespace gnt {

constexpr int kNumCUs = 256;
constexpr int64_t kMaxLeadingDim = (int64_t)1 << 22;   // keeps tile byte offsets below 2^31
constexpr int64_t kDefaultWorkspaceMB = 128;

struct Config {
    const char *name;
    int bm, bn, bk, waves, stages;
    int lds;        // LDS bytes per workgroup
    int kmask;      // zeroes operand columns past K in registers (any K)
    int splitk;     // supports splits > 1
};

// The kernel family.  The kernel-template tiles use stages * (BM + BN) * BK * 2
// bytes of LDS (at most 160 KB) and give each wave a (BM/WM) x (BN/WN) block of
// 32x32 MFMA tiles.  Configurations with kmask = 1 zero the operand columns past
// K in registers and are the only ones planned when K is not a multiple of 8.
inline const Config kConfigs[] = {
    {"128x128x64_w8_s4", 128, 128, 64, 8, 4, 131072, 0, 1},
    {"128x128x64_w8_s4_kmask", 128, 128, 64, 8, 4, 131072, 1, 1},
    {"256x256x64_w8_pp2", 256, 256, 64, 8, 9, 147456, 0, 1},
    {"128x128x64_w8_s2", 128, 128, 64, 8, 2, 65536, 0, 1},
    {"32x128x64_w4_s6", 32, 128, 64, 4, 6, 122880, 0, 1},
    {"256x128x64_w4_u8", 256, 128, 64, 4, 8, 163840, 0, 1},
};
constexpr int kNumConfigs = sizeof(kConfigs) / sizeof(kConfigs[0]);
enum {
    CFG_T128x128 = 0,
    CFG_T128x128_KMASK = 1,
    CFG_PP2_256x256 = 2,
    CFG_T128x128_S2 = 3,
    CFG_T32x128 = 4,
    CFG_W4_256x128 = 5,
};

struct Plan {
    int cfg;
    int stream;            // stream-K: the persistent ping-pong kernel + streamk_sum
    int sk_maxseg;         // stream-K partial slots per block
    int64_t sk_units;      // stream-K units, tiles * k_tiles
    int tiles_m, tiles_n;
    int k_tiles;
    int splits;
    int kt_per_split;
    int group_m;
    int64_t grid;
    int64_t ws_bytes;
    int inreduce;          // two K splits reduced inside the kernel (no second pass)
};

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Whether the tile kernels (32x128, 128x128) walk their k-slabs in the
// rotated order (SlabOrder; `mode` as GEMM_ROTATE).  Rotation spreads the
// blocks' row offsets over the memory channels, which pays where B streams
// from HBM and A is small (M <= 128: 1 x 4096 x 16384 38.0 -> 28.3 us,
// 127 x 28672 x 8192 102.6 -> 95.4, 1 x 8192 x 8192 30.0 -> 28.2).  With 256
// rows of A that every tile reads, tiles at different slabs no longer share
// A's slabs in L2 as they go (256 x 8192 x 8192 on the four-wave tile: 57.3
// -> 62.3 us), and on the large shapes it measured level or slower, so the
// 256-row tiles always walk K in order.
inline bool rotate_slabs(int mode, int64_t M) { return mode == 2 || (mode == 1 && M <= 128); }

inline int find_config(const char *name)
{
    for (int i = 0; i < kNumConfigs; ++i)
        if (strcmp(kConfigs[i].name, name) == 0)
            return i;
    return -1;
}

// Pick the tile shape and the K split for a problem.  `ws_bytes` bounds the
// split-K partial storage; `force_cfg` / `force_splits` (>= 0 / > 0) override.
inline Plan make_plan(int64_t M, int64_t N, int64_t K, int64_t ws_bytes, int force_cfg, int force_splits,
               int streamk = 0, int inreduce = 1)
{
    Plan p{};
    int cfg;
    // A tile family's blocks with the K splits the split rule below would give
    // it (at least min_slabs 64-deep slabs each), and the fraction of their
    // passes of the machine they fill.
    const int64_t kt64 = cdiv(K, 64);
    auto blocks = [&](int64_t tiles, int64_t min_slabs) {
        int64_t s = 1;
        if (tiles < kNumCUs && kt64 >= 16)
            s = std::max<int64_t>(1, std::min<int64_t>(kNumCUs / tiles, kt64 / min_slabs));
        return tiles * s;
    };
    auto fill = [](int64_t b) { return (double)b / (double)(cdiv(b, kNumCUs) * kNumCUs); };
    if (force_cfg >= 0) {
        cfg = force_cfg;
    } else if (K % 8) {
        cfg = CFG_T128x128_KMASK;
    } else if (M <= 64) {
        // The 32x128 tile, while its tiles fit one pass of the machine: two
        // 32-row tiles per column still beat one 128-row tile at 64 x 4096 x
        // 4096 (15.3 against 20.8 us) and are level with it at 40 x 8192 x 8192
        // (32.3 against 32.5).  Past one pass (M > 32 over N > 16384) the
        // second, mostly empty pass costs more than the 128-row tile's idle
        // rows: 40 x 28672 x 8192 73.9 against 103.2 us, 64 x 28672 x 8192 77.0
        // against 110.9.  From M = 96 the 128x128 tile is faster by half.
        cfg = M <= 32 || cdiv(M, 32) * cdiv(N, 128) <= kNumCUs ? CFG_T32x128 : CFG_T128x128;
    } else if (M <= 128) {
        cfg = CFG_T128x128;
    } else if (M <= 256) {
        // Decode batches: the whole of M in one 256-row tile of the ping-pong
        // kernel (A stays in L2, every compute unit streams its own 256-row
        // panel of B), and split-K below to bring the grid up to the machine.
        // When that tile would need more than four K splits (few N tiles:
        // 256 x 10240 x 8192, 256 x 8192 x 8192, 256 x 8192 x 28672), the
        // four-wave 256 x 128 tile fills the machine with half as many splits,
        // i.e. half the FP32 partial traffic (interleaved medians: 59.5 -> 56.6,
        // 53.0 -> 50.0, 126.2 -> 123.0 us; with two splits, at 256 x 28672 x
        // 8192, the ping-pong tile stays faster: 122.6 against 126.1 us).
        //
        // Either 256-row tile only while its blocks fill the machine as well
        // as the 128x128 tile's would (the fraction of the passes they fill,
        // with the K splits the split rule below gives each): with short K or
        // few N tiles the 256-row tiles' splits (at least 20 slabs each) leave
        // most compute units idle.  Interleaved medians: 192 x 4096 x 4096
        // 22.4 us on the 128x128 tile against 42.8 on the ping-pong tile,
        // 256 x 8192 x 2048 21.7 against 41.6, 256 x 2048 x 8192 26.5 against 33.9 on the four-wave tile; and
        // the four-wave tile over the ping-pong one when it fills more
        // (256 x 16384 x 4096: 45.3 against 53.0 us), or as much while the
        // ping-pong tile's splits would hold fewer than 64 slabs each
        // (256 x 28672 x 4096: 62.7 against 67.1 us; at K = 8192, 64 slabs
        // per split, the ping-pong tile: 121.8 against 124.3).
        cfg = CFG_PP2_256x256;
        const int64_t t256 = cdiv(N, 256);
        const int64_t s256 = std::min<int64_t>(kNumCUs / std::max<int64_t>(1, t256), kt64 / 20);
        const int64_t b_w4 = blocks(cdiv(N, 128), 20), b_128 = blocks(cdiv(M, 128) * cdiv(N, 128), 8);
        const int64_t b_pp2 = blocks(t256, 20);
        double f = fill(b_pp2);
        const bool short_splits = kt64 * t256 / b_pp2 < 64;
        if (t256 < kNumCUs && (s256 > 4 || fill(b_w4) > f || (fill(b_w4) == f && short_splits))) {
            cfg = CFG_W4_256x128;
            f = fill(b_w4);
        }
        if (fill(b_128) > f)
            cfg = CFG_T128x128;
    } else {
        // The 256x256 ping-pong tile when its blocks fill at least half the
        // machine, with the K splits the split rule below would give it (at
        // least 20 k-slabs each); smaller tiles otherwise.
        const int64_t big = std::max<int64_t>(1, cdiv(M, 256) * cdiv(N, 256));
        const int64_t ksplit = std::min<int64_t>(kNumCUs / big, cdiv(K, 64) / 20);
        cfg = big * std::max<int64_t>(1, ksplit) >= kNumCUs / 2 ? CFG_PP2_256x256 : CFG_T128x128;
        // ... and the 128x128 tile even then, when its tiles fit one pass and
        // fill it at least as well (640 x 2048 x 8192: 37.9 against 50.6 us;
        // 768 x 4096 x 4096 40.9 against 44.5; 384 x 8192 x 4096 41.9 against
        // 45.6).  Its plans past one pass (the two-stage ring) measured mixed
        // against the ping-pong tile and keep the rule above.
        const int64_t t128 = cdiv(M, 128) * cdiv(N, 128);
        if (cfg == CFG_PP2_256x256 && t128 < kNumCUs && fill(blocks(t128, 8)) >= fill(blocks(big, 20)))
            cfg = CFG_T128x128;
    }
    // The 32x128 tile wherever the 128x128 tile was chosen above M = 64 but
    // the 32-row tiles, in one pass with their own K splits, fill the machine
    // strictly better: small squares and small problems with short K.  On
    // the small ragged shapes it takes, the two tiles, each with its own K
    // splits, measured level (178 x 640 x 2240: 11.0 us both; 74 x 1408 x
    // 512 8.8; 618 x 704 x 3968 16.4 against 16.3), where the plans that
    // earlier rules made for them took 16.6, 11.2 and 19.8 us.  On a tie
    // the 128x128 tile, whose blocks do more work per byte staged.
    if (cfg == CFG_T128x128 && M > 64) {
        const int64_t t32 = cdiv(M, 32) * cdiv(N, 128), t128 = cdiv(M, 128) * cdiv(N, 128);
        if (t32 <= kNumCUs && fill(blocks(t32, 8)) > fill(blocks(t128, 8)))
            cfg = CFG_T32x128;
    }
    // 128x128 tiles that overflow one pass of the machine but fit two: the
    // two-stage ring (64 KB of LDS) lets two blocks share a compute unit, so
    // they all run at once instead of leaving a second, nearly empty wave.
    if (cfg == CFG_T128x128 && force_cfg < 0) {
        const int64_t t128 = cdiv(M, 128) * cdiv(N, 128);
        if (t128 > kNumCUs && t128 <= 2 * kNumCUs)
            cfg = CFG_T128x128_S2;
    }
    if ((K % 8) && !kConfigs[cfg].kmask)
        cfg = CFG_T128x128_KMASK;
    const Config &c = kConfigs[cfg];
    p.cfg = cfg;
    p.tiles_m = (int)cdiv(M, c.bm);
    p.tiles_n = (int)cdiv(N, c.bn);
    p.k_tiles = (int)cdiv(K, c.bk);
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;

    int splits = 1;
    if (!c.splitk) {
        splits = 1;
    } else if (force_splits > 0) {
        splits = force_splits;
    } else if (tiles < kNumCUs && (int64_t)p.k_tiles * c.bk >= 16 * 64) {
        // Fill the compute units, keeping at least 512 of K per split (1280
        // for the 256x256 tiles, whose 256 KB FP32 partial per split costs as
        // much as streaming about 256 of K of B).
        // For M <= 32 the 32-row tile's blocks each stream their own rows of
        // B, once: with a block on every compute unit those streams measured
        // up to 60% slower than with about three quarters of them (more
        // concurrent DRAM streams, not more bytes), so the split count aims
        // there, rounded to the nearest.
        const int min_slabs = (c.bm == 256 ? 20 : 8) * 64 / c.bk;
        if (cfg == CFG_T32x128 && M <= 32)
            splits = (int)((3 * kNumCUs / 4 + tiles / 2) / tiles);
        else
            splits = (int)(kNumCUs / tiles);
        if (splits > p.k_tiles / min_slabs)
            splits = p.k_tiles / min_slabs;
        if (splits < 1)
            splits = 1;
    }
    // For M <= 32 the 32-row tile streams B rows whose K splits start
    // kt_per_split * 128 bytes apart.  Starts a multiple of 4 KB apart measured
    // up to 20% slower (the blocks of one B row then hit the same DRAM channels
    // together), so the nearest split count with another stride is taken.
    // Only when the fill rule split K: with one split no two blocks start in
    // the same B row.
    if (cfg == CFG_T32x128 && M <= 32 && force_splits <= 0 && p.k_tiles >= 16 && splits > 1) {
        auto aliased = [&](int sp) { return (cdiv(p.k_tiles, sp) * c.bk * 2) % 4096 == 0; };
        auto ok = [&](int sp) { return sp >= 1 && sp <= 8 && p.k_tiles / sp >= 8 && !aliased(sp); };
        if (aliased(splits)) {
            for (int d = 1; d < 8; ++d) {
                if (ok(splits - d)) {
                    splits -= d;
                    break;
                }
                if (ok(splits + d)) {
                    splits += d;
                    break;
                }
            }
        }
    }
    while (splits > 1 && (int64_t)splits * M * N * 4 > ws_bytes)
        --splits;
    if (p.k_tiles == 0)
        splits = 1;
    if (splits > p.k_tiles && p.k_tiles > 0)
        splits = p.k_tiles;
    p.kt_per_split = splits > 1 ? (int)cdiv(p.k_tiles, splits) : p.k_tiles;
    if (splits > 1)
        splits = (int)cdiv(p.k_tiles, p.kt_per_split);   // no empty split
    p.splits = splits;
    p.group_m = p.tiles_m >= 4 ? 4 : p.tiles_m;
    if (p.group_m < 1)
        p.group_m = 1;
    p.grid = tiles * splits;
    p.ws_bytes = splits > 1 ? (int64_t)splits * M * N * 4 : 0;
    // Two K splits on the 256-row tiles, any number on the tile kernels with a
    // ring deeper than two stages: the last split of a tile to finish adds the
    // others' partials (one BM x BN FP32 slot per split and tile) and stores
    // the tile, instead of a second pass over [splits][M][N] partials.
    const bool many = cfg != CFG_PP2_256x256 && cfg != CFG_W4_256x128 && c.stages > 2;
    const bool two = cfg == CFG_PP2_256x256 || cfg == CFG_W4_256x128;
    if (inreduce && ((splits == 2 && two) || (splits >= 2 && many)) &&
        tiles * 4 <= GEMM_COUNTER_BYTES) {
        const int64_t need = tiles * splits * (int64_t)c.bm * c.bn * 4;
        if (need <= ws_bytes) {
            p.inreduce = 1;
            p.ws_bytes = need;
        }
    }

    // Stream-K (the CuTe page's section 9 names it beside split-K): when the
    // ping-pong tiles with their K splits leave at least 3/8 of the compute
    // units idle, every unit takes an equal run of the tiles * k_tiles
    // (tile, k-slab) units instead, each tile it touches giving one partial
    // (a 256 KB slot).  Only for runs of at least 32 k-slabs: each segment
    // refills the pipeline and writes a whole partial tile, which shorter runs
    // do not pay back.  `streamk`: 0 never, 1 by this rule (the default), 2
    // whenever the tile is the ping-pong one.  Interleaved medians on operands
    // read cold: 3000 x 3000 x 5000 (144 tiles) 126 us against 141 without;
    // 2304 x 2304 x 8192 (three splits fill the machine) 130 against 88;
    // 3000 x 3000 x 1536 (runs of 13 slabs) 70 against 50.  With operands
    // resident in the memory-side cache the first one reverses (125 against
    // 118): stream-K pays where the idle compute units would add HBM streams.
    if (streamk > 0 && cfg == CFG_PP2_256x256 && force_splits <= 0 && tiles > 0 && p.k_tiles > 0) {
        const int64_t T = tiles * p.k_tiles;
        const int64_t G = std::min<int64_t>(kNumCUs, T);
        const int64_t L = (T + G - 1) / G;                 // longest run
        const int maxseg = (int)((L - 1) / p.k_tiles + 2);
        const int64_t ws = G * maxseg * (int64_t)256 * 256 * 4;
        const bool idle = p.grid * 8 <= (int64_t)kNumCUs * 5;
        if (ws <= ws_bytes && T < INT32_MAX && (streamk == 2 || (idle && L >= 32))) {
            p.stream = 1;
            p.sk_units = T;
            p.sk_maxseg = maxseg;
            p.splits = 1;
            p.kt_per_split = p.k_tiles;
            p.grid = G;
            p.ws_bytes = ws;
        }
    }
    return p;
}

}  // namespace gnt
