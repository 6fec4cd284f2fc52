// rows_group.hpp -- grouping of index entries: n entries, each naming one of G
// groups (anything else: none), give the groups' counts, their offsets and the
// entries' stable order.  A first launch (which may make the ids, too) counts each
// block's entries, a last one places them (place_block), each block after what
// the blocks before it place.  That is added up by every placing block for
// itself while there are few blocks, else by a launch in between (scan_column):
// 257 columns of 256 blocks took 33 us when each placing block added them up.
// Counts are integers, so the LDS atomics' order does not show; places come from
// ranks, not from atomics.
#pragma once

#include "rows_common.hpp"

namespace gnt {

constexpr int kMaxGroups = 1024;
constexpr int kGroupThreads = 1024;
constexpr int kGroupWaves = kGroupThreads / 64;

// A block's group counts in LDS to hist[block][G + 1] (entry G: no group).
__device__ __forceinline__ void store_hist(const int *lds_hist, int *hist, int G)
{
    for (int e = threadIdx.x; e <= G; e += blockDim.x)
        hist[(int64_t)blockIdx.x * (G + 1) + e] = lds_hist[e];
}

// LDS of place_block.
struct PlaceLds {
    int start[kMaxGroups + 1];     // group's offset plus what earlier blocks place there
    int wave[kGroupWaves][kMaxGroups + 1];   // each wave's own counts, then its first place
    int part[kGroupWaves];
};

// Exclusive prefix sums of v[0 .. count), in place, by all threads (at most
// 2 * kGroupThreads values); returns the total.
__device__ __forceinline__ int scan_lds(int *v, int count, int *part)
{
    constexpr int PER = 2;
    static_assert(PER * kGroupThreads >= kMaxGroups + 1, "one pass");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int x[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = tid * PER + i;
        x[i] = at < count ? v[at] : 0;
        sum += x[i];
    }
    int run = sum;
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(run, o);
        if (lane >= o)
            run += y;
    }
    if (lane == 63)
        part[wave] = run;
    __syncthreads();
    int before = run - sum, total = 0;
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) {
        if (w < wave)
            before += part[w];
        total += part[w];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int at = tid * PER + i;
        if (at < count)
            v[at] = before;
        before += x[i];
    }
    __syncthreads();
    return total;
}

// The launch in between: this block's 64 columns of the counts, one column a lane,
// the waves taking the rows (counting blocks) in turn.  hist[b][e] becomes what
// the blocks before b place in e, totals[e] the whole.
__device__ __forceinline__ void scan_column(int *hist, int *totals, int G, int blocks, int (&part)[kGroupWaves][64])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e = blockIdx.x * 64 + lane;
    const int b0 = (int)((int64_t)wave * blocks / kGroupWaves), b1 = (int)((int64_t)(wave + 1) * blocks / kGroupWaves);
    int sum = 0;
    if (e <= G)
#pragma unroll 8
        for (int b = b0; b < b1; ++b)
            sum += hist[(int64_t)b * (G + 1) + e];
    part[wave][lane] = sum;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < wave; ++w)
        before += part[w][lane];
    if (e <= G) {
#pragma unroll 8
        for (int b = b0; b < b1; ++b) {
            int *at = hist + (int64_t)b * (G + 1) + e;
            const int c = *at;
            *at = before;
            before += c;
        }
        if (wave == kGroupWaves - 1)
            totals[e] = before;
    }
}

// Block b of `blocks`, each of `chunk` entries: offsets, counts (block 0 writes
// them) and the places of this block's entries.  kGroupThreads threads.
// SCANNED: hist and totals are scan_column's.
template <bool SCANNED>
__device__ __forceinline__ void place_block(PlaceLds &l, const int32_t *ids, int64_t n, int G, int64_t chunk,
                                            const int *hist, const int *totals, int b, int blocks,
                                            int32_t *counts, int32_t *offsets, int32_t *order)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // counts of all blocks, and of the blocks before this one
    for (int e = tid; e <= G; e += kGroupThreads) {
        if constexpr (SCANNED) {
            l.start[e] = totals[e];
            l.wave[0][e] = hist[(int64_t)b * (G + 1) + e];
        } else {
            int before = 0, total = 0;
#pragma unroll 8
            for (int i = 0; i < blocks; ++i) {
                const int c = hist[(int64_t)i * (G + 1) + e];
                before += i < b ? c : 0;
                total += c;
            }
            l.start[e] = total;
            l.wave[0][e] = before;
        }
    }
    __syncthreads();
    if (b == 0)
        for (int e = tid; e < G; e += kGroupThreads)
            counts[e] = l.start[e];
    __syncthreads();
    scan_lds(l.start, G + 1, l.part);
    for (int e = tid; e <= G; e += kGroupThreads) {
        if (b == 0)
            offsets[e] = l.start[e];       // entry G: what the groups hold together
        l.start[e] += l.wave[0][e];
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kGroupWaves; ++w)
        for (int e = tid; e <= G; e += kGroupThreads)
            l.wave[w][e] = 0;
    __syncthreads();
    // this wave's stretch of the block's entries, 64 at a time
    const int64_t c0 = (int64_t)b * chunk, c1 = c0 + chunk < n ? c0 + chunk : n;
    const int64_t per = (chunk + kGroupThreads - 1) / kGroupThreads * 64;
    const int64_t w0 = c0 + wave * per, w1 = w0 + per < c1 ? w0 + per : c1;
    auto group_of = [&](int64_t i) {
        const int g = i < w1 ? ids[i] : -1;
        return (uint32_t)g < (uint32_t)G ? g : G;
    };
    for (int64_t i = w0 + lane; i < w1; i += 64)
        atomicAdd(&l.wave[wave][group_of(i)], 1);
    __syncthreads();
    for (int e = tid; e <= G; e += kGroupThreads) {
        int at = l.start[e];
#pragma unroll
        for (int w = 0; w < kGroupWaves; ++w) {
            const int c = l.wave[w][e];
            l.wave[w][e] = at;
            at += c;
        }
    }
    __syncthreads();
    const int bits = 32 - __builtin_clz(G);   // of the group numbers 0 .. G
    for (int64_t i0 = w0; i0 < w1; i0 += 64) {
        const int64_t i = i0 + lane;
        const bool in = i < w1;
        const int g = group_of(i);
        // the lanes with this lane's group, from one ballot per bit of the number
        uint64_t same = __builtin_amdgcn_ballot_w64(in);
        for (int k = 0; k < bits; ++k) {
            const uint64_t ones = __builtin_amdgcn_ballot_w64((g >> k) & 1);
            same &= (g >> k) & 1 ? ones : ~ones;
        }
        const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
        int at = 0;
        if (in)
            at = l.wave[wave][g] + rank;
        __builtin_amdgcn_wave_barrier();
        if (in) {
            order[at] = (int32_t)i;
            if (rank == 0)                       // the group's first lane moves its place on
                l.wave[wave][g] = at + __builtin_popcountll(same);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

}  // namespace gnt
