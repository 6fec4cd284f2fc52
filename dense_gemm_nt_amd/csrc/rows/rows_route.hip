// rows_route.hip -- the top-k router: softmax, choices, per-expert counts and
// order, balance loss; and its gradient.
//
// A token's logits are spread over LPR lanes of 4 Q columns each (from column
// 4 Q li for lane li), so a row is read once and held in registers: maximum, sum
// and the k choices come from reductions over the LPR lanes.  A choice is one
// maximum over the lanes and a ballot for its first holder, so ties fall to the
// lowest column.  Up to 64 experts several rows share a wave and a choice is worked
// out in vector registers (route_rows_narrow); with more a wave has one row, each
// lane its columns sorted, so that a choice compares one value a lane: the maximum
// is a scalar, its holder a scalar search in one ballot (route_rows_wide), about 22
// vector operations a choice, where maxima over all of a lane's columns and ballots
// for each took about 45.
//
// 65536 x 256 FP32, 8 choices: forward 49 us (67 MB; 366 vector operations
// a row bound it), counts' scan 10, places 10, gradient 39 (141 MB, 3.6 TB/s).  16 x
// 64, the one launch of a small call: 9.4 us, all of it round trips and reductions.
#include <type_traits>

#include "rows_group.hpp"
#include "rows_host.hpp"

namespace gnt {
namespace {

enum : int { L_BF16 = 0, L_FP16 = 1, L_FP32 = 2 };

struct RouteArgs {
    const void *logits;
    const uint8_t *mask;
    int64_t T, ld;
    int E, k, renorm, vec;
    int64_t per_block;        // tokens of a block
    int blocks;
    int32_t *ids;
    float *weights;
    int32_t *counts, *offsets, *order, *tokens;
    float *loss;
    int *hist;                // [blocks][E + 1]
    float *psum;              // [blocks][E]
    int *live;                // [blocks]
    int *totals;              // [E + 1]
    float *loss_part;         // [(E + 64) / 64]
    // backward
    const float *grad_w, *grad_loss;
    void *dlogits;
    int64_t ldd;
    int vec_d;
};

template <int CTRL>
__device__ __forceinline__ float dpp(float x)
{
    // (every lane has a source under these patterns; said so, the move folds into its use)
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

// x combined over the LPR lanes of a row, in every one of them.
template <int LPR, typename F>
__device__ __forceinline__ float over_row(float x, F op)
{
    if constexpr (LPR >= 2)
        x = op(x, dpp<0xB1>(x));       // lanes 1 apart
    if constexpr (LPR >= 4)
        x = op(x, dpp<0x4E>(x));       // 2 apart
    if constexpr (LPR >= 8)
        x = op(x, dpp<0x141>(x));      // the other quad of eight
    if constexpr (LPR >= 16)
        x = op(x, dpp<0x140>(x));      // the other eight of sixteen
    if constexpr (LPR >= 32) {
        const unsigned v = __builtin_bit_cast(unsigned, x);
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        const unsigned lo = r[0], hi = r[1];   // (values: a bit cast of an element takes the first)
        x = op(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi));
    }
    if constexpr (LPR >= 64) {
        const unsigned v = __builtin_bit_cast(unsigned, x);
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        const unsigned lo = r[0], hi = r[1];   // (values: a bit cast of an element takes the first)
        x = op(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi));
    }
    return x;
}

template <int LPR>
__device__ __forceinline__ float row_max(float x)
{
    return over_row<LPR>(x, [](float a, float b) { return fmaxf(a, b); });
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x)
{
    return over_row<LPR>(x, [](float a, float b) { return a + b; });
}

// Four consecutive values of a row from column c; past E: -inf.
template <int DT>
__device__ __forceinline__ f32x4 load_logits(const void *base, int64_t row, int c, int E, int vec)
{
    f32x4 x;
    if constexpr (DT == L_FP32) {
        const float *p = static_cast<const float *>(base) + row + c;
        if (vec && c + 4 <= E)
            return *reinterpret_cast<const f32x4 *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = c + i < E ? p[i] : -INFINITY;
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(base) + row + c;
        uint16_t h[4];
        if (vec && c + 4 <= E) {
            const u32x2 w = *reinterpret_cast<const u32x2 *>(p);
            h[0] = (uint16_t)w[0], h[1] = (uint16_t)(w[0] >> 16);
            h[2] = (uint16_t)w[1], h[3] = (uint16_t)(w[1] >> 16);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = from16<DT>(h[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = c + i < E ? from16<DT>(p[i]) : -INFINITY;
        }
    }
    return x;
}

template <int DT>
__device__ __forceinline__ void store_logits(void *base, int64_t row, int c, int E, int vec, f32x4 x)
{
    if constexpr (DT == L_FP32) {
        float *p = static_cast<float *>(base) + row + c;
        if (vec && c + 4 <= E) {
            *reinterpret_cast<f32x4 *>(p) = x;
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < E)
                p[i] = x[i];
    } else {
        uint16_t *p = static_cast<uint16_t *>(base) + row + c;
        if (vec && c + 4 <= E) {
            u32x2 w;
            w[0] = (uint32_t)to16<DT>(x[0]) | ((uint32_t)to16<DT>(x[1]) << 16);
            w[1] = (uint32_t)to16<DT>(x[2]) | ((uint32_t)to16<DT>(x[3]) << 16);
            *reinterpret_cast<u32x2 *>(p) = w;
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < E)
                p[i] = to16<DT>(x[i]);
    }
}

// e^d for d <= 0, NaN for NaN: 2^(d log2 e), with what the rounding of that product left put
// back to first order.  Without it the result is off by 2^-24 for each unit of d: at
// d = -80, 2^-18.  (An infinite d has no such rest; below -200 all is zero anyway.)
__device__ __forceinline__ float exp_below(float d)
{
    constexpr float log2e = 1.44269504088896340736, ln2 = 0.69314718055994530942;
    constexpr float log2e_rest = 1.44269504088896340736 - (double)log2e;
    d = d < -200.0f ? -200.0f : d;
    const float t = d * log2e;
    const float rest = __builtin_fmaf(d, log2e_rest, __builtin_fmaf(d, log2e, -t));
    const float r = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(r * rest, ln2, r);
}

// A row's softmax from its logits: p in place of x; false for a row without an
// open expert.  key is the ranking value of each logit (NaN as the lowest
// finite one).
template <int LPR, int Q>
__device__ __forceinline__ bool softmax_row(f32x4 (&x)[Q], f32x4 (&key)[Q])
{
    float top = -INFINITY;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            key[q][i] = x[q][i] != x[q][i] ? -3.402823466e38f : x[q][i];
            top = fmaxf(top, key[q][i]);
        }
    top = row_max<LPR>(top);
    const bool open = top > -INFINITY;
    top = open ? top : 0.0f;           // (a closed row's exponentials are then zeros)
    float sum = 0.0f;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[q][i] = exp_below(x[q][i] - top);
            sum += x[q][i];
        }
    sum = row_sum<LPR>(sum);
    const float inv = open ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[q][i] *= inv;
    return open;
}

// The balance loss of n routed tokens from s = sum_e counts_e psum_e.
__device__ __forceinline__ void write_loss(const RouteArgs &a, int n, float s)
{
    const float nf = (float)n;
    *a.loss = n > 0 ? (float)a.E * (s / nf) / (nf * (float)a.k) : 0.0f;
    *a.tokens = n;
}

// The balance loss from counts (a function of e) and the routed tokens' sums of p.
template <typename P, typename C>
__device__ __forceinline__ void balance_loss(const RouteArgs &a, int n, P psum, C count, float *red)
{
    float part = 0.0f;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x)
        part += (float)count(e) * psum(e);
    part = row_sum<64>(part);
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = part;
    __syncthreads();
    if (threadIdx.x == 0) {
        float s = 0.0f;
        for (int w = 0; w < (int)(blockDim.x >> 6); ++w)
            s += red[w];
        write_loss(a, n, s);
    }
}

// Integers in the order of the floats (-0 is made +0); NaN as the lowest finite
// value.
__device__ __forceinline__ int rank_key(float x)
{
    const int b = __builtin_bit_cast(int, x != x ? -3.402823466e38f : x + 0.0f);
    return b ^ ((b >> 31) & 0x7fffffff);
}
constexpr int kClosedKey = (int)0x807fffffu;     // rank_key(-inf); a taken column is below it

__device__ __forceinline__ float rank_value(int k)
{
    return __builtin_bit_cast(float, k ^ ((k >> 31) & 0x7fffffff));
}

// The largest of a wave's values, as a scalar.
__device__ __forceinline__ int wave_max(int x)
{
    x = max(x, __builtin_amdgcn_mov_dpp(x, 0xB1, 0xf, 0xf, true));
    x = max(x, __builtin_amdgcn_mov_dpp(x, 0x4E, 0xf, 0xf, true));
    x = max(x, __builtin_amdgcn_mov_dpp(x, 0x141, 0xf, 0xf, true));
    x = max(x, __builtin_amdgcn_mov_dpp(x, 0x140, 0xf, 0xf, true));
    int a = max(__builtin_amdgcn_readlane(x, 0), __builtin_amdgcn_readlane(x, 16));
    int b = max(__builtin_amdgcn_readlane(x, 32), __builtin_amdgcn_readlane(x, 48));
    asm("" : "+s"(a), "+s"(b));        // (kept apart, or they become a vector maximum of three)
    return max(a, b);
}

// One wave's walk over its rows, one at a time.  `sum` collects p, hist (in LDS)
// the choices; returns how many of the wave's rows were routed.
template <int DT, int Q, int NW>
__device__ __forceinline__ int route_rows_wide(const RouteArgs &a, int64_t t0, int64_t t1, int wave, int lane,
                                               f32x4 (&sum)[Q], int *hist)
{
    constexpr int V = 4 * Q, BITS = Q == 1 ? 2 : Q == 2 ? 3 : 4;
    typedef std::conditional_t<Q == 4, uint64_t, uint32_t> order_t;
    const int64_t mine = t0 + wave;
    // (the mask is not waited for: a masked row is loaded like any other)
    f32x4 next[Q];
    uint8_t next_on = 1;
    auto load = [&](int64_t t) {
        if (t >= t1)
            return;
        if (a.mask)
            next_on = a.mask[t];
#pragma unroll
        for (int q = 0; q < Q; ++q)
            next[q] = load_logits<DT>(a.logits, t * a.ld, lane * V + 4 * q, a.E, a.vec);
    };
    constexpr bool AHEAD = Q < 4;        // (16 columns a lane leave no registers for it)
    int routed = 0;
    if constexpr (AHEAD)
        load(mine);
    for (int64_t t = mine; t < t1; t += NW) {
        if constexpr (!AHEAD)
            load(t);
        f32x4 x[Q];
        int key[V], at[V];
        const bool on = __builtin_amdgcn_readfirstlane(next_on) != 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float value = next[v / 4][v % 4];
            x[v / 4][v % 4] = value;
            key[v] = rank_key(value);
            at[v] = v;
        }
        if constexpr (AHEAD)
            load(t + NW);               // the next row's loads run under this row
        int found = 0, my_e = -1, my_key = 0;
        float inv = 0.0f, top = 0.0f;
        int best = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v)
            best = max(best, key[v]);
        best = on ? wave_max(best) : kClosedKey;
        if (best > kClosedKey) {
            ++routed;
            top = rank_value(best);
            float total = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                x[v / 4][v % 4] = exp_below(x[v / 4][v % 4] - top);
                total += x[v / 4][v % 4];
            }
            inv = 1.0f / row_sum<64>(total);
#pragma unroll
            for (int q = 0; q < Q; ++q)
                sum[q] += x[q] * inv;
            // the lane's columns by falling key, by odd-even transposition: neighbours
            // only change places where they must, so equal ones stay in order
#pragma unroll
            for (int r = 0; r < V; ++r)
#pragma unroll
                for (int v = r & 1; v + 1 < V; v += 2) {
                    const bool swap = key[v + 1] > key[v];
                    const int hi = max(key[v], key[v + 1]), lo = min(key[v], key[v + 1]);
                    const int i = swap ? at[v + 1] : at[v], j = swap ? at[v] : at[v + 1];
                    key[v] = hi, key[v + 1] = lo, at[v] = i, at[v + 1] = j;
                }
            // ... and the columns in that order, BITS bits each
            order_t order = 0;
#pragma unroll
            for (int v = V - 1; v >= 0; --v)
                order = order << BITS | (order_t)at[v];
            // (best: the largest value left)
            for (;;) {
                // its first holder, and that lane's next column
                const uint64_t has = __builtin_amdgcn_ballot_w64(key[0] == best);
                const int l = __builtin_ctzll(has);
                const int e = l * V + (__builtin_amdgcn_readlane((int)order, l) & (V - 1));
                my_e = lane == found ? e : my_e;
                my_key = lane == found ? best : my_key;
                if (++found == a.k)
                    break;
                // (masks, not selections: those of array elements became searches)
                const int holder = lane == l ? -1 : 0;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    key[v] = ((v + 1 < V ? key[v + 1] : INT32_MIN) & holder) | (key[v] & ~holder);
                order >>= holder & BITS;
                best = wave_max(key[0]);
                if (best <= kClosedKey)
                    break;
            }
        }
        // lane j holds choice j: its weight from its logit, as p was made
        const bool chose = lane < found;
        float w = chose ? exp_below(rank_value(my_key) - top) * inv : 0.0f;
        if (a.renorm && found)
            w /= row_sum<64>(w);        // (a division: a single choice's weight is 1, not nearly 1)
        if (lane < a.k) {
            a.ids[t * a.k + lane] = my_e;
            a.weights[t * a.k + lane] = w;
            atomicAdd(&hist[chose ? my_e : a.E], 1);
        }
    }
    return routed;
}

// GPW rows at a time, LPR lanes each; counts a row in its first lane.
template <int DT, int LPR, int NW>
__device__ __forceinline__ int route_rows_narrow(const RouteArgs &a, int64_t t0, int64_t t1, int wave, int lane,
                                                 f32x4 (&sum)[1], int *hist)
{
    constexpr int GPW = 64 / LPR;
    const int li = lane % LPR, grp = lane / LPR;
    int routed = 0;
    for (int64_t base = t0 + wave * GPW; base < t1; base += NW * GPW) {
        const int64_t t = base + grp;
        const bool in = t < t1;
        const f32x4 closed = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        f32x4 x[1], key[1];
        x[0] = in ? load_logits<DT>(a.logits, t * a.ld, li * 4, a.E, a.vec) : closed;
        if (a.mask && in)               // (after the row's own load, which does not wait for it)
            x[0] = a.mask[t] ? x[0] : closed;
        const bool open = softmax_row<LPR, 1>(x, key);
        routed += open && li == 0;
        sum[0] += x[0];
        uint8_t place_of[4] = {0xff, 0xff, 0xff, 0xff};
        float chosen = 0.0f;
        int found = 0;
        for (int j = 0; j < a.k; ++j) {
            float best = fmaxf(fmaxf(key[0][0], key[0][1]), fmaxf(key[0][2], key[0][3]));
            best = row_max<LPR>(best);
            const bool more = best > -INFINITY;
            if (__builtin_amdgcn_ballot_w64(more) == 0)
                break;
            found += more;
            const bool mine = more && (key[0][0] == best || key[0][1] == best || key[0][2] == best ||
                                       key[0][3] == best);
            const uint64_t row = (__builtin_amdgcn_ballot_w64(mine) >> (grp * LPR)) & ((1ull << LPR) - 1);
            if (mine && __builtin_ctzll(row) == li) {
                bool taken = false;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!taken && key[0][i] == best) {
                        taken = true;
                        key[0][i] = -INFINITY;
                        place_of[i] = (uint8_t)j;
                        chosen += x[0][i];
                    }
            }
        }
        chosen = row_sum<LPR>(chosen);
        const float share = a.renorm && found ? chosen : 1.0f;
        if (in) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (place_of[i] != 0xff) {
                    const int e = li * 4 + i;
                    a.ids[t * a.k + place_of[i]] = e;
                    a.weights[t * a.k + place_of[i]] = x[0][i] / share;
                    atomicAdd(&hist[e], 1);
                }
            for (int j = found + li; j < a.k; j += LPR) {
                a.ids[t * a.k + j] = -1;
                a.weights[t * a.k + j] = 0.0f;
                atomicAdd(&hist[a.E], 1);
            }
        }
    }
    return routed;
}

// One block of tokens: choices, weights, the block's counts and sums of p.
// ONE: the only block, which then also finishes (counts, order, loss).
template <int DT, int LPR, int Q, bool ONE>
__global__ __launch_bounds__(kGroupThreads) void route_forward(RouteArgs a)
{
    constexpr int NW = kGroupThreads / 64, COLS = LPR * 4 * Q;
    __shared__ int hist[kMaxGroups + 1];
    __shared__ float ps[NW][COLS];
    __shared__ int live[NW];
    __shared__ std::conditional_t<ONE, PlaceLds, int> place;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane % LPR, grp = lane / LPR;
    for (int e = tid; e <= a.E; e += kGroupThreads)
        hist[e] = 0;
    __syncthreads();

    const int64_t t0 = blockIdx.x * a.per_block;
    const int64_t t1 = t0 + a.per_block < a.T ? t0 + a.per_block : a.T;
    f32x4 sum[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
        sum[q] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    int routed;
    if constexpr (LPR == 64) {
        routed = route_rows_wide<DT, Q, NW>(a, t0, t1, wave, lane, sum, hist);
    } else {
        routed = route_rows_narrow<DT, LPR, NW>(a, t0, t1, wave, lane, sum, hist);
        for (int o = 32; o; o >>= 1)
            routed += __shfl_xor(routed, o);
    }
    // the block's sums of p: over the rows of a wave, then over the waves
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v = sum[q][i];
            for (int o = LPR; o < 64; o <<= 1)
                v += __shfl_xor(v, o);
            if (grp == 0)
                ps[wave][li * 4 * Q + 4 * q + i] = v;
        }
    if (lane == 0)
        live[wave] = routed;
    __syncthreads();
    auto psum = [&](int e) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w)
            v += ps[w][e];
        return v;
    };
    int n = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w)
        n += live[w];
    store_hist(hist, a.hist, a.E);
    if constexpr (ONE) {
        balance_loss(a, n, psum, [&](int e) { return hist[e]; }, reinterpret_cast<float *>(place.part));
        __syncthreads();
        place_block<false>(place, a.ids, a.T * a.k, a.E, a.per_block * a.k, a.hist, nullptr, 0, 1, a.counts,
                           a.offsets, a.order);
    } else {
        for (int e = tid; e < a.E; e += kGroupThreads)
            a.psum[(int64_t)blockIdx.x * a.E + e] = psum(e);
        if (tid == 0)
            a.live[blockIdx.x] = n;
    }
}

// The second launch of a larger batch: 64 experts a block, what each forward
// block places and the experts' part of the loss sum_e counts_e psum_e, the
// blocks' sums of p added in order.
__global__ __launch_bounds__(kGroupThreads) void route_scan(RouteArgs a)
{
    __shared__ int part[kGroupWaves][64];
    __shared__ float sums[kGroupWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e = blockIdx.x * 64 + lane;
    const int b0 = (int)((int64_t)wave * a.blocks / kGroupWaves), b1 = (int)((int64_t)(wave + 1) * a.blocks / kGroupWaves);
    float v = 0.0f;
    if (e < a.E)
#pragma unroll 8
        for (int b = b0; b < b1; ++b)
            v += a.psum[(int64_t)b * a.E + e];
    sums[wave][lane] = v;
    scan_column(a.hist, a.totals, a.E, a.blocks, part);     // (a barrier between)
    if (wave == 0) {
        float p = 0.0f;
        int c = 0;
        for (int w = 0; w < kGroupWaves; ++w) {
            p += sums[w][lane];
            c += part[w][lane];
        }
        const float s = row_sum<64>(e < a.E ? (float)c * p : 0.0f);
        if (lane == 0)
            a.loss_part[blockIdx.x] = s;
    }
}

// The third: counts, offsets, order; the loss (a block more than the entries').
__global__ __launch_bounds__(kGroupThreads) void route_place(RouteArgs a)
{
    __shared__ PlaceLds place;
    if ((int)blockIdx.x < a.blocks) {
        place_block<true>(place, a.ids, a.T * a.k, a.E, a.per_block * a.k, a.hist, a.totals, blockIdx.x, a.blocks,
                          a.counts, a.offsets, a.order);
        return;
    }
    int n = 0;
    for (int i = threadIdx.x; i < a.blocks; i += kGroupThreads)
        n += a.live[i];
    for (int o = 32; o; o >>= 1)
        n += __shfl_xor(n, o);
    if ((threadIdx.x & 63) == 0)
        place.part[threadIdx.x >> 6] = n;
    __syncthreads();
    if (threadIdx.x == 0) {
        n = 0;
        for (int w = 0; w < kGroupWaves; ++w)
            n += place.part[w];
        float s = 0.0f;
        for (int i = 0; i < (a.E + 64) / 64; ++i)
            s += a.loss_part[i];
        write_loss(a, n, s);
    }
}

// dlogit = p (dp - sum p dp), dp_e = g_loss E f_e / n + (the gradient of e's
// weight, if chosen): p is recomputed from the logits, which are read once.  Lane j
// of a row takes choice j's gradient, and LDS carries it to the lane that holds
// the expert's column (a wave's own 256 Q values: no barrier).  Renormalized
// weights' gradients are h_j = (g_j - sum_i g_i w_i) / S with sum_i w_i = 1: they are taken as
// ((g_j - g_0) - sum_i (g_i - g_0) w_i) / S, which does not leave the rounding of
// sum_i w_i times g where w_0 is nearly 1 or the only weight (it was 1e-7 of g / S then, in
// FP32 1.5e-5 of dlogits with the loss's gradient beside it).
template <int DT, int LPR, int Q>
__global__ __launch_bounds__(256) void route_backward(RouteArgs a)
{
    constexpr int GPW = 64 / LPR, COLS = LPR * 4 * Q;
    __shared__ __attribute__((aligned(16))) float chosen[4][GPW][COLS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int li = lane % LPR, grp = lane / LPR;
    float *mine = chosen[wave][grp];
    const float n = (float)*a.tokens;
    const float gl = a.grad_loss && n > 0.0f ? *a.grad_loss * (float)a.E / (n * n * (float)a.k) : 0.0f;
    f32x4 from_loss[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = li * 4 * Q + 4 * q + i;
            from_loss[q][i] = e < a.E ? gl * (float)a.counts[e] : 0.0f;
        }
    const int64_t step = (int64_t)gridDim.x * 4 * GPW;
    const bool vec = a.vec;
    auto load = [&](int64_t t, f32x4 (&x)[Q]) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
            x[q] = t < a.T ? load_logits<DT>(a.logits, t * a.ld, li * 4 * Q + 4 * q, a.E, vec)
                           : (f32x4){-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    };
    f32x4 next[Q];
    const int64_t first = ((int64_t)blockIdx.x * 4 + wave) * GPW + grp;
    load(first, next);
    for (int64_t t = first; t - grp < a.T; t += step) {
        const bool in = t < a.T;
        const bool on = in && a.ids[t * a.k] >= 0;     // a routed token has a first choice
        f32x4 x[Q], key[Q], dp[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q)
            x[q] = on ? next[q] : (f32x4){-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        load(t + step, next);
        softmax_row<LPR, Q>(x, key);
#pragma unroll
        for (int q = 0; q < Q; ++q)
            dp[q] = from_loss[q];
        if (a.grad_w) {
            const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
            auto wave_sync = [] {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_wave_barrier();
            };
            float mean = 0.0f, inv = 1.0f, g0 = 0.0f;
            if (a.renorm) {
                g0 = on ? a.grad_w[t * a.k] : 0.0f;
                // p where the choices are: their sum, and sum of (g - g_0) w
#pragma unroll
                for (int q = 0; q < Q; ++q)
                    *reinterpret_cast<f32x4 *>(mine + li * 4 * Q + 4 * q) = x[q];
                wave_sync();
                float total = 0.0f;
                for (int j = li; j < a.k; j += LPR) {
                    const int e = on ? a.ids[t * a.k + j] : -1;
                    if ((uint32_t)e < (uint32_t)a.E) {
                        total += mine[e];
                        mean += (a.grad_w[t * a.k + j] - g0) * a.weights[t * a.k + j];
                    }
                }
                total = row_sum<LPR>(total);
                mean = row_sum<LPR>(mean);
                inv = total != 0.0f ? 1.0f / total : 1.0f;
                wave_sync();
            }
#pragma unroll
            for (int q = 0; q < Q; ++q)
                *reinterpret_cast<f32x4 *>(mine + li * 4 * Q + 4 * q) = zero;
            wave_sync();
            for (int j = li; j < a.k; j += LPR) {
                const int e = on ? a.ids[t * a.k + j] : -1;
                if ((uint32_t)e < (uint32_t)a.E)
                    mine[e] = (a.grad_w[t * a.k + j] - g0 - mean) * inv;
            }
            wave_sync();
#pragma unroll
            for (int q = 0; q < Q; ++q)
                dp[q] += *reinterpret_cast<const f32x4 *>(mine + li * 4 * Q + 4 * q);
            wave_sync();
        }
        float dot = 0.0f;
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                dot += x[q][i] * dp[q][i];
        dot = row_sum<LPR>(dot);
        if (in)
#pragma unroll
            for (int q = 0; q < Q; ++q)
                store_logits<DT>(a.dlogits, t * a.ldd, li * 4 * Q + 4 * q, a.E, a.vec_d, x[q] * (dp[q] - dot));
    }
}

// At most two blocks for every compute unit: all of them at once.
int64_t tokens_per_block(int64_t T)
{
    return std::max<int64_t>(cdiv(cdiv(T, 2 * kNumCUs), 16) * 16, 64);
}

template <typename F>
gemm_status_t by_width(int E, F launch)
{
    if (E <= 16)
        launch(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
    else if (E <= 64)
        launch(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
    else if (E <= 256)
        launch(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    else if (E <= 512)
        launch(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
    else
        launch(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
    return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

template <typename F>
gemm_status_t by_type(int dtype, int E, F launch)
{
    if (dtype == GEMM_BF16)
        return by_width(E, [&](auto l, auto q) { launch(std::integral_constant<int, L_BF16>{}, l, q); });
    if (dtype == GEMM_FP16)
        return by_width(E, [&](auto l, auto q) { launch(std::integral_constant<int, L_FP16>{}, l, q); });
    return by_width(E, [&](auto l, auto q) { launch(std::integral_constant<int, L_FP32>{}, l, q); });
}

gemm_status_t check_route(int64_t T, int64_t E, int64_t k)
{
    if (T < 0 || E < 0 || k < 0)
        return GEMM_ERR_INVALID_ARG;
    if (E < 1 || E > kMaxGroups || k < 1 || k > E || k > 64 || T >= kMaxSize || T * k >= kMaxSize)
        return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

// four values of a row as one load: every row starts aligned to it
bool rows_vectorize(const void *p, int64_t ld, int dtype)
{
    return (uintptr_t)p % (4 * size_of(dtype)) == 0 && ld % 4 == 0;
}

void carve_route(Carver &c, RouteArgs &a)
{
    a.hist = c.take<int>((int64_t)a.blocks * (a.E + 1));
    a.psum = c.take<float>((int64_t)a.blocks * a.E);
    a.live = c.take<int>(a.blocks);
    a.totals = c.take<int>(a.E + 1);
    a.loss_part = c.take<float>((a.E + 64) / 64);
}

}  // namespace
}  // namespace gnt

using namespace gnt;

extern "C" {

gemm_status_t gemm_route_workspace(int64_t T, int64_t E, int64_t top_k, int64_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_INVALID_ARG;
    *bytes = 0;
    const gemm_status_t st = check_route(T, E, top_k);
    if (st != GEMM_OK)
        return st;
    RouteArgs a{};
    a.E = (int)E;
    a.blocks = (int)std::max<int64_t>(1, cdiv(T, tokens_per_block(T)));
    Carver c{nullptr};
    carve_route(c, a);
    *bytes = c.used;
    return GEMM_OK;
}

gemm_status_t gemm_run_route(const void *logits, const uint8_t *mask, int64_t T, int64_t E,
                             int64_t ld, int64_t top_k, int renormalize, int dtype,
                             const gemm_routing_t *out, void *workspace, int64_t workspace_bytes,
                             hipStream_t stream)
{
    gemm_status_t st = check_route(T, E, top_k);
    if (st != GEMM_OK)
        return st;
    if (!is_out(dtype) || ld >= kMaxSize)
        return GEMM_ERR_UNSUPPORTED;
    if (ld < E || !out || !out->counts || !out->offsets || !out->tokens || !out->loss ||
        (T > 0 && (!logits || !out->ids || !out->weights || !out->order)))
        return GEMM_ERR_INVALID_ARG;
    for (const void *p : {(const void *)out->ids, (const void *)out->weights, (const void *)out->counts,
                          (const void *)out->offsets, (const void *)out->order, (const void *)out->tokens,
                          (const void *)out->loss})
        if ((uintptr_t)p % 4)
            return GEMM_ERR_MISALIGNED;
    if ((uintptr_t)logits % size_of(dtype))
        return GEMM_ERR_MISALIGNED;
    RouteArgs a{};
    a.logits = logits;
    a.mask = mask;
    a.T = T;
    a.ld = ld;
    a.E = (int)E;
    a.k = (int)top_k;
    a.renorm = renormalize != 0;
    a.vec = rows_vectorize(logits, ld, dtype);
    a.per_block = tokens_per_block(T);
    a.blocks = (int)std::max<int64_t>(1, cdiv(T, a.per_block));
    a.ids = out->ids;
    a.weights = out->weights;
    a.counts = out->counts;
    a.offsets = out->offsets;
    a.order = out->order;
    a.tokens = out->tokens;
    a.loss = out->loss;
    Carver c{static_cast<uint8_t *>(workspace)};
    carve_route(c, a);
    if ((st = check_workspace(workspace, workspace_bytes, c.used)) != GEMM_OK)
        return st;
    const bool one = a.blocks == 1;
    st = by_type(dtype, a.E, [&](auto dt, auto lpr, auto q) {
        if (one)
            hipLaunchKernelGGL((route_forward<dt.value, lpr.value, q.value, true>), dim3(1), dim3(kGroupThreads),
                               0, stream, a);
        else
            hipLaunchKernelGGL((route_forward<dt.value, lpr.value, q.value, false>), dim3(a.blocks),
                               dim3(kGroupThreads), 0, stream, a);
    });
    if (st != GEMM_OK || one)
        return st;
    hipLaunchKernelGGL(route_scan, dim3((unsigned)((E + 64) / 64)), dim3(kGroupThreads), 0, stream, a);
    hipLaunchKernelGGL(route_place, dim3(a.blocks + 1), dim3(kGroupThreads), 0, stream, a);
    return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

gemm_status_t gemm_run_route_backward(const void *logits, const gemm_routing_t *in,
                                      const float *grad_weights, const float *grad_loss,
                                      void *dlogits, int64_t T, int64_t E, int64_t ld, int64_t ldd,
                                      int64_t top_k, int renormalize, int dtype,
                                      hipStream_t stream)
{
    const gemm_status_t st = check_route(T, E, top_k);
    if (st != GEMM_OK)
        return st;
    if (!is_out(dtype) || ld >= kMaxSize || ldd >= kMaxSize)
        return GEMM_ERR_UNSUPPORTED;
    if (ld < E || ldd < E || !in)
        return GEMM_ERR_INVALID_ARG;
    if (T == 0)
        return GEMM_OK;
    if (!logits || !dlogits || !in->ids || !in->weights || !in->counts || !in->tokens)
        return GEMM_ERR_INVALID_ARG;
    if ((uintptr_t)logits % size_of(dtype) || (uintptr_t)dlogits % size_of(dtype) ||
        (uintptr_t)grad_weights % 4 || (uintptr_t)grad_loss % 4 || (uintptr_t)in->ids % 4 ||
        (uintptr_t)in->weights % 4 || (uintptr_t)in->counts % 4 || (uintptr_t)in->tokens % 4)
        return GEMM_ERR_MISALIGNED;
    RouteArgs a{};
    a.logits = logits;
    a.T = T;
    a.ld = ld;
    a.E = (int)E;
    a.k = (int)top_k;
    a.renorm = renormalize != 0;
    a.vec = rows_vectorize(logits, ld, dtype);
    a.ids = in->ids;
    a.weights = in->weights;
    a.counts = in->counts;
    a.tokens = in->tokens;
    a.grad_w = grad_weights;
    a.grad_loss = grad_loss;
    a.dlogits = dlogits;
    a.ldd = ldd;
    a.vec_d = rows_vectorize(dlogits, ldd, dtype);
    return by_type(dtype, a.E, [&](auto dt, auto lpr, auto q) {
        constexpr int rows = 4 * 64 / lpr.value;       // of a block and pass
        const unsigned grid = (unsigned)std::min<int64_t>(cdiv(T, rows), 2048);
        hipLaunchKernelGGL((route_backward<dt.value, lpr.value, q.value>), dim3(grid), dim3(256), 0, stream, a);
    });
}

}  // extern "C"
