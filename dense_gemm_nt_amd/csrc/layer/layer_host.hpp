// layer_host.hpp -- plans, workspaces and launches that the layer's entry points share (host
// code).
#pragma once

#include "gemm_layer.h"
#include "../rows/rows_host.hpp"
#include "layer_common.hpp"

namespace gnt {

constexpr int64_t kPartialBytes = (int64_t)64 << 20;   // bound on a plan's K-split partials

// A product's partials and arrival counters in a workspace.
struct SplitWs {
    float *partials;
    unsigned *counters;
    int num_counters;
};

inline SplitWs carve_splits(Carver &c, const Plan &p)
{
    SplitWs w;
    w.num_counters = p.inreduce ? p.tiles_m * p.tiles_n : 0;
    w.partials = c.take<float>(p.splits > 1 ? p.ws_bytes / 4 : 0);
    w.counters = c.take<unsigned>(w.num_counters);
    return w;
}

// The tile's arguments from its plan (operands and sizes that only the caller knows are
// set by it).
inline void fill_args(KernelArgs &a, const Plan &p, const SplitWs &w, void *C, int64_t M, int64_t N, int64_t K,
                      int64_t ldc, int out_dtype)
{
    const int64_t size = size_of(out_dtype);
    a.C = C;
    a.M = (int)M, a.N = (int)N, a.K = (int)K;
    a.ldc = (int)ldc;
    a.tiles_m = p.tiles_m, a.tiles_n = p.tiles_n;
    a.k_tiles = p.k_tiles;
    a.splits = p.splits;
    a.kt_per_split = p.kt_per_split;
    a.group_m = p.group_m;
    a.vec_store = ldc % 4 == 0 && (uintptr_t)C % (4 * size) == 0;
    a.rows16 = (ldc * size) % 16 == 0 && (uintptr_t)C % 16 == 0;
    a.nt_b = p.tiles_m <= 2;
    a.partials = w.partials;
    a.counters = w.counters;
    a.inreduce = p.inreduce;
    a.alpha = 1.0f;
}

// What a plan's launches are expected to take, in us, M x N: the passes over the machine of a
// beginning and its slabs each, and the partials of K splits at 4 TB/s (less where the kernel sums
// them: they meet in an L2).  From sweeps of tiles and splits during development (K in elements of
// 16 bits; us, predicted / measured): 200 x 10240 x 4096 four-wave tile 3 splits 43 / 43, 128 x 128 1
// split 36 / 43, ping-pong 6 splits 54 / 46; 512 x 8192 x 4096 128 x 128 36 / 45, ping-pong 4 splits
// 70 / 56; 400 x 16384 x 4096 four-wave 62 / 65, ping-pong 2 splits 78 / 78; 1500 x 10928 x 4096
// ping-pong 204 / 187, 128 x 128 179 / 186.  So the 128 x 128 tile is taken to be up to a fifth faster
// than it is, and ping-pong plans with splits up to a quarter slower: the order of the plans of
// 129 to 2000 rows is only as good as that (the 8-bit product's slabs were measured at 0.57 us on
// the 128 x 128 tile, and have the 16-bit ones' 0.45 here).
inline double plan_us(const Plan &p, int64_t M, int64_t N)
{
    const double per = p.kt_per_split;
    const double passes = (double)cdiv(p.grid, kNumCUs);
    const double partials = p.splits > 1 ? (double)p.splits * (double)M * (double)N * 8.0 / 4e6 : 0.0;
    const double sum = p.splits <= 1 ? 0.0 : p.inreduce ? 4.0 + 0.7 * partials : 4.0 + partials;
    switch (p.cfg) {
    case CFG_PP2_256x256: return passes * (9.0 + 1.45 * per) + sum;
    case CFG_W4_256x128: return passes * (9.0 + 0.82 * per) + sum;
    case CFG_T32x128: return passes * (6.0 + 0.35 * per) + sum;
    case CFG_T128x128_S2: return (double)cdiv(p.grid, 2 * kNumCUs) * (7.0 + (p.grid > kNumCUs ? 1.0 : 0.6) * per) + sum;
    default: return passes * (7.0 + 0.45 * per) + sum;
    }
}

// A product's plan: the NT library's, or above 128 rows the 128 x 128 tile or the four-wave one
// where it is expected to take a tenth less (512 x 8192 x 4096 45 us against 55; 256 x 8192 x 4096 35 against
// 39; 700 x 10240 x 4096 66 against 83; 300 x 10928 x 4096 62 against 71).
inline Plan plan_product(int64_t M, int64_t N, int64_t K)
{
    const Plan p = make_plan(M, N, K, kPartialBytes, -1, -1, 0);
    if (M <= 128)
        return p;
    Plan best = p;
    double least = 0.9 * plan_us(p, M, N);
    for (int cfg : {(int)CFG_T128x128, (int)CFG_W4_256x128})
        for (int splits : {-1, 1}) {
            const Plan q = make_plan(M, N, K, kPartialBytes, cfg, splits, 0);
            const double us = plan_us(q, M, N);
            if (us < least)
                least = us, best = q;
        }
    return best;
}

// A product in one launch, or in two: where the ping-pong tiles' last pass over the machine would be
// mostly empty, the rows (or columns) of the whole passes, and then the rest on a plan of its
// own.  8111 x 8200 x 4096 (1056 tiles, 33 in a row) 523 us in one launch, whose fifth pass has 32,
// 450 in two; 1500 x 10928 x 4096 (258 tiles) 185, and 138 as 42 columns of tiles and the rest.
struct Pieces {
    struct {
        int64_t row, rows, col, cols;
        Plan plan;
    } at[2];
    int count;
};

inline Pieces plan_pieces(int64_t M, int64_t N, int64_t K)
{
    Pieces best{};
    best.at[0] = {0, M, 0, N, plan_product(M, N, K)};
    best.count = 1;
    const Plan big = make_plan(M, N, K, kPartialBytes, CFG_PP2_256x256, 1, 0);
    if (big.cfg != CFG_PP2_256x256 || big.grid <= kNumCUs)
        return best;
    double least = 0.95 * plan_us(best.at[0].plan, M, N);
    const int64_t whole = big.grid / kNumCUs * kNumCUs;
    for (bool by_cols : {false, true}) {
        const int64_t cut = whole / (by_cols ? big.tiles_m : big.tiles_n) * 256, end = by_cols ? N : M;
        if (cut == 0 || cut >= end)
            continue;
        Pieces t{};
        t.count = 2;
        const int64_t m0 = by_cols ? M : cut, n0 = by_cols ? cut : N;
        const int64_t m1 = by_cols ? M : M - cut, n1 = by_cols ? N - cut : N;
        t.at[0] = {0, m0, 0, n0, make_plan(m0, n0, K, kPartialBytes, CFG_PP2_256x256, 1, 0)};
        t.at[1] = {by_cols ? 0 : cut, m1, by_cols ? cut : 0, n1, plan_product(m1, n1, K)};
        const double us = plan_us(t.at[0].plan, m0, n0) + 2.0 + plan_us(t.at[1].plan, m1, n1);
        if (us < least)
            least = us, best = t;
    }
    return best;
}

inline bool launchable(const Plan &p) { return p.grid > 0 && p.grid < kMaxBlocks; }

// Zeros to the arrival counters of up to four products (a kernel: a captured fill of
// another kind has given wrong results on replays).
hipError_t clear_counters(const SplitWs *w, int count, hipStream_t stream);

}  // namespace gnt
