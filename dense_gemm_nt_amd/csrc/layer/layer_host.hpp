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

inline bool launchable(const Plan &p) { return p.grid > 0 && p.grid < kMaxBlocks; }

// Zeros to the arrival counters of up to three products (a kernel: a captured fill of
// another kind has given wrong results on replays).
hipError_t clear_counters(const SplitWs *w, int count, hipStream_t stream);

}  // namespace gnt
