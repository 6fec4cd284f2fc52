// rows_common.hpp -- pieces shared by the kernels whose weight depends on the
// row: argument blocks, conversions, the walk over a row block's adapters.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../gemm_nt_common.hpp"

namespace gnt {

// A projection with low-rank adapters: the tile's arguments plus the adapters.
// low holds, in K split s's plane of low_stride values, row m's unscaled low-rank
// product (its part) at m * rank_pad; up is [adapter][N][rank] (adapter a at
// a * up_stride elements, rows of up_ld elements).
struct LoraArgs : KernelArgs {
    const float *low;
    const uint16_t *up;
    const float *scale;
    const int32_t *ids;
    int64_t up_stride;
    int64_t low_stride;
    int up_ld;
    int adapters;          // 0: no adapters, nothing is added
    int rank, rank_pad;    // rank_pad: rank rounded up to 16
    int low_splits;
};

// Products over rows sorted by expert.  A, B, C (and lda, ldb, ldc) are the whole
// arrays; every block finds its expert, hence its tile, from the offsets.
struct RoutedArgs : KernelArgs {
    const int32_t *offsets;   // [experts + 1]
    int experts;
    int rows;                 // of the sorted arrays
    int tile_m;               // rows (weight gradient: rows of dW_e) of a tile
    int tail;                 // rows of no expert (before the first's, behind the last's)
                              // are set to zero
    int wgrad;                // dW_e [N][K] = dY_e^T X_e, else C_e = X_e op(W_e)
    int64_t b_stride;         // elements between experts' W
    int64_t c_stride;         // wgrad: elements between experts' dW
    int c_size;               // bytes of an element of C
};

// v combined with the lanes below it, inclusively.
template <typename F>
__device__ __forceinline__ int wave_scan(int v, int lane, F op)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(v, o);
        v = lane >= o ? op(v, y) : v;
    }
    return v;
}

// Block id -> its tile's expert, and the expert's problem and tile within it;
// false for a block past the last tile.  The grid is the host's bound on the
// tiles (which it does not know).  Every wave scans the offsets by itself, 64
// experts at a time, stopping at its own: about a microsecond for up to 64
// experts, where a launch of its own to write a problem list costs several.
// Offsets are read clamped to [0, rows] and to their running maximum, so that
// whatever they hold no row outside the arrays is touched.
//
// Launch order: block ids go round-robin over the 8 XCDs, and the ids of one
// XCD take runs of 32 consecutive tiles (its compute units) within every 256,
// so that tiles sharing panels meet in one L2; the order does not depend on the
// number of tiles, so the blocks without one are spread over the XCDs.
__device__ __forceinline__ bool routed_lookup(RoutedArgs &p, int &tm, int &tn)
{
    const int lane = threadIdx.x & 63;
    const int bid = blockIdx.x;
    const int v = (bid & ~255) + (bid & 7) * 32 + ((bid >> 3) & 31);
    const int E = p.experts, rows = p.rows;
    auto at = [&](int e) { return min(max(p.offsets[e], 0), rows); };
    int top = 0, before = 0;                 // carried over the experts scanned
    for (int e0 = 0; e0 <= E + 1; e0 += 64) {
        const int e = e0 + lane;
        const int lo = e <= E ? at(e) : 0, hi = e < E ? at(e + 1) : 0;
        const int most = max(top, wave_scan(lo, lane, [](int a, int b) { return max(a, b); }));
        // entry E is the rows behind the last expert's, entry E + 1 those before the first's
        const int start = e <= E ? most : 0;
        const int count = e < E ? max(start, hi) - start : !p.tail ? 0 : e == E ? rows - start : e == E + 1 ? at(0) : 0;
        const int tall = p.wgrad ? (e < E ? p.M : 0) : count;
        const int tiles = ((tall + p.tile_m - 1) / p.tile_m) * p.tiles_n;
        const int past = before + wave_scan(tiles, lane, [](int a, int b) { return a + b; });
        const uint64_t holds = __builtin_amdgcn_ballot_w64(v < past);
        if (holds) {
            const int l = __builtin_ctzll(holds);
            const int g = e0 + l;
            const int s = __builtin_amdgcn_readlane(start, l), n = __builtin_amdgcn_readlane(count, l);
            const int t = v - (__builtin_amdgcn_readlane(past, l) - __builtin_amdgcn_readlane(tiles, l));
            p.A += (int64_t)s * p.lda;
            if (p.wgrad) {
                p.B += (int64_t)s * p.ldb;
                p.C = static_cast<uint8_t *>(p.C) + (int64_t)g * p.c_stride * p.c_size;
                p.K = n;
            } else {
                p.B += (int64_t)(g < E ? g : 0) * p.b_stride;
                p.C = static_cast<uint8_t *>(p.C) + (int64_t)s * p.ldc * p.c_size;
                p.M = n;
                p.K = g < E ? p.K : 0;       // rows of no expert: a sum over nothing
            }
            p.tiles_m = (p.M + p.tile_m - 1) / p.tile_m;
            p.k_tiles = (p.K + 63) / 64;
            p.splits = 1;
            p.kt_per_split = p.k_tiles;
            p.nt_b = p.tiles_m <= 2;
            tile_order(t, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
            return true;
        }
        top = __builtin_amdgcn_readlane(most, 63);
        before = __builtin_amdgcn_readlane(past, 63);
    }
    return false;
}

template <int IN>
__device__ __forceinline__ uint16_t to16(float x)
{
    if constexpr (IN == IN_BF16)
        return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
    else
        return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
}

template <int IN>
__device__ __forceinline__ float from16(uint16_t h)
{
    if constexpr (IN == IN_BF16)
        return static_cast<float>(__builtin_bit_cast(__bf16, h));
    else
        return static_cast<float>(__builtin_bit_cast(_Float16, h));
}

// An FP32 value as the sum of NP 16-bit ones, for the matrix cores: each the nearest to what
// the ones before it leave.  Two bf16 values are within 2^-17 of x relative to it, two
// fp16 ones within 2^-23 from 2^-2 on and 2^-25 absolute below (fp16's steps no longer shrink
// below 2^-14: the caller keeps x up), where one value would be within 2^-8 or 2^-11.  The
// low-rank products are intermediates that the caller never sees: rounding them to 16 bits would
// put an error into the output that nothing else in it has.  A result of 16 bits does not
// show what two leave (a 64th of its own half step at most); an FP32 one of BF16 operands
// does, and takes three (low_parts).  Each costs an MFMA per rank-16 step, of which an output
// tile has rank / 16 beside its K / 16.  An infinite part (an infinity, or past fp16's
// range) stands alone.
template <int IN, int NP>
__device__ __forceinline__ void split16(float x, uint16_t (&part)[NP])
{
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        part[i] = to16<IN>(x);
        const float h = from16<IN>(part[i]);
        x = __builtin_isfinite(h) ? x - h : 0.0f;
    }
}

template <int IN, int OUT>
constexpr int low_parts = IN == IN_BF16 && OUT == OUT_FP32 ? 3 : 2;

// The same for the gradients' contraction over rows, whose FP32 results keep what
// their operands hold: three bf16 parts, 24 bits, whatever the operands' type (with
// two the adapters' gradients were 2.5e-6 off, with three as near as FP32 sums
// are).  bf16 has FP32's range: two fp16 parts lose what is below 2^-25, and with it all of
// a beginning adapter's gradients (dy and B of 1e-4: 12% off), and end at 65504.  So
// FP16 operands are multiplied in bf16 as well, as two parts themselves
// (bf16_halves).  The second of those is not multiplied with the third part (2^-26 of the
// product), so a value that is not finite is held there alone: an infinity never meets
// a second half of zero.  The low-rank values and gradients of 8192 rows, 12288 columns,
// rank 32 take 115 us of FP16 operands and 100 of BF16 ones.
constexpr int kParts = 3;

__device__ __forceinline__ void split_parts(float x, uint16_t (&part)[kParts])
{
    const uint16_t hi = to16<IN_BF16>(x);
    const bool finite = (hi & 0x7f80u) != 0x7f80u;
    const float r = x - from16<IN_BF16>(hi);
    const uint16_t mid = to16<IN_BF16>(r);
    part[0] = finite ? hi : 0;
    part[1] = finite ? mid : 0;
    part[2] = finite ? to16<IN_BF16>(r - from16<IN_BF16>(mid)) : hi;
}

// What add_special takes as the first part of values held as split_parts makes them.
__device__ __forceinline__ u32x4 first_part(const u32x4 (&part)[kParts])
{
    u32x4 y;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t x = part[kParts - 1][d];
        y[d] = part[0][d] | ((x & 0x7f80u) == 0x7f80u ? x & 0xffffu : 0u) |
               ((x & 0x7f800000u) == 0x7f800000u ? x & 0xffff0000u : 0u);
    }
    return y;
}

// Eight finite fp16 values as sums of two bf16 ones, exactly: of 11 bits the first 8
// (the FP32 value cut off) and the 3 left, in bf16's wider range.
__device__ __forceinline__ void bf16_halves(u32x4 x, u32x4 &hi, u32x4 &lo)
{
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        uint32_t h[2], l[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float v = from16<IN_FP16>((uint16_t)(x[d] >> (16 * i)));
            h[i] = __builtin_bit_cast(uint32_t, v) & 0xffff0000u;
            l[i] = __builtin_bit_cast(uint32_t, v - __builtin_bit_cast(float, h[i]));
        }
        hi[d] = h[0] >> 16 | h[1];
        lo[d] = l[0] >> 16 | (l[1] & 0xffff0000u);
    }
}

template <int IN>
__device__ __forceinline__ f32x4 mfma16x16x32(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (IN == IN_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Wait states between a loop of MFMAs and what reads their results by other
// units.  The compiler places these itself, but was seen to leave them out where
// the loop's end and a path around the loop meet before an LDS store (the stored
// values were then those of some cycles before); after such loops they are
// placed here.  24 states cover the longest MFMA used (19).
__device__ __forceinline__ void mfma_settle()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15\n\ts_nop 7" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Nonzero where one of eight 16-bit values is an infinity or NaN: an exponent of
// all ones carries into the sign's place when one is added to it.
template <int IN>
__device__ __forceinline__ uint32_t has_special(u32x4 x)
{
    constexpr uint32_t one = IN == IN_BF16 ? 0x00800080u : 0x04000400u;
    uint32_t c = 0;
#pragma unroll
    for (int d = 0; d < 4; ++d)
        c |= (x[d] & 0x7fff7fffu) + one;
    return c & 0x80008000u;
}

// Each 16-bit value v of a fragment replaced by f(v).
template <typename F>
__device__ __forceinline__ u32x4 each16(u32x4 x, F f)
{
    u32x4 y;
#pragma unroll
    for (int d = 0; d < 4; ++d)
        y[d] = f(x[d] & 0xffffu) | f(x[d] >> 16) << 16;
    return y;
}

// acc += x . v where x holds infinities or NaNs, and v is held as several parts: as the
// sum of x's finite values (its others as +-1 to 2, by their exponents' highest bit: an
// infinite v then stays one, and a NaN a NaN; finite(x) multiplies them by all parts)
// and of what its others make, from v's first part hi, without any operand that could make a zero of
// another row, or of a later part, into a NaN.  +-2^127 times +-2^127 (bf16) overflows to the infinity
// that is due and is 0 where hi is masked to 0; a NaN (also that of infinity times 0) is
// made as the sum of both infinities.  Where not `own`, v's parts are zeros that
// are to add nothing.  mul(x, y) multiplies bf16 values and adds to acc.  Rarely run, and
// written for few registers: one operand pair at a time.
template <int IN, typename P, typename F>
__device__ __forceinline__ void add_special(u32x4 x, u32x4 hi, bool own, P finite, F mul)
{
    constexpr uint32_t exp = IN == IN_BF16 ? 0x7f80u : 0x7c00u, big = 0x7f00u;
    auto step = [&](auto f, auto g, uint32_t flip) {
        mul(each16(x, f), each16(hi, g) ^ flip);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto is_nan = [](uint32_t v) { return (v & 0x7fffu) > exp ? big : 0u; };
    auto is_inf = [](uint32_t v) { return (v & 0x7fffu) == exp ? big : 0u; };
    auto inf = [](uint32_t v) { return (v & 0x7fffu) == exp ? (v & 0x8000u) | big : 0u; };
    auto sign = [](uint32_t v) { return v & 0x7fffu ? (v & 0x8000u) | big : 0u; };
    const uint32_t mine = own ? big : 0u;
    auto all = [&](uint32_t) { return mine; };
    auto zero = [&](uint32_t v) { return v & 0x7fffu ? 0u : mine; };
    {
        constexpr uint32_t exps = exp << 16 | exp, lowest = exps & ~(exps << 1);
        u32x4 y;
#pragma unroll
        for (int d = 0; d < 4; ++d)
            y[d] = x[d] & ~((((x[d] & exps) + lowest) & 0x80008000u) >> 1);
        finite(y);
        __builtin_amdgcn_sched_barrier(0);
    }
    step(inf, sign, 0u);
    step(is_nan, all, 0u);
    step(is_nan, all, 0x80008000u);
    step(is_inf, zero, 0u);
    step(is_inf, zero, 0x80008000u);
}

// Adds every row's low-rank part to a wave's accumulators:
//   acc[m][n] += s_a sum_r low[m][r] up_a[n][r],  a = ids[m]
// for the 32 FM rows from r0 and 32 FN columns from c0, in the accumulators'
// own layout (the up rows are the MFMA's first operand), so the shared
// projection's sum is rounded once, together with the adapters'.  The wave walks the
// adapters of its rows (a scalar walk over ballots: any order of rows, no
// sorting), and for each the rows of other adapters enter as zeros: an adapter's
// up rows are read once by every wave that has a row of it.  (Zero times an
// infinity or NaN among those up rows would reach the other rows: adapters
// whose fragments hold one are taken apart, add_special.)  A tile's K splits
// share its adapters, split s taking the adapters s, s + splits, ... of each
// wave's walk, so that all of a decode grid's blocks stream them; NB adapters'
// fragments are in flight together, and AHEAD the next ranks' low-rank values (as
// the tile leaves registers for).  Rows without an adapter, and ids that name
// none, add nothing.  Nothing here waits on the tile's own loads.
//
// fp16 parts of a low-rank value hold its bits only between 2^-3 and 2^15.  A row whose
// largest value of a rank step lies outside has its accumulators and the values in units of a
// power of two from then on, in which that value is just below 2^15 (2^-60 to 2^60: an
// accumulator of FP16 products is below 2^63, so its units keep it in FP32's range), and
// they are turned back at the end: multiplications by powers of two, in the rare tile.  A
// value is then off by 2^-22 of its step's largest at most, or 2^-40 of the row's largest
// in the steps before.
// Without it a value of 2^-25 was lost and one of 2^16 infinite, also in FP32 results.
// The projection's kernel with adapters and with ids that name none: 4096 x 8192 x 8192,
// rank 64, 4 adapters in runs 450 us against 398; 64 x 10240 x 8192, rank 16, 48
// adapters 48.3 against 37.0; 1 x 4096 x 4096, rank 16 13.5 against 12.4.  What it adds is
// the round trips of ids, low-rank values and up rows, one after the other, at the end of
// a tile.
template <int IN, int NB, bool AHEAD, int NP, int FN, int FM>
__device__ __forceinline__ void lora_add(const LoraArgs &p, f32x16 (&acc)[FN][FM], int r0, int c0, int split,
                                         int lane)
{
    if (p.adapters == 0 || r0 >= p.M || c0 >= p.N)
        return;
    int id[FM];
    uint32_t rows[FM];
    uint32_t any = 0;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
        const int m = r0 + fm * 32 + (lane & 31);
        const int a = m < p.M ? p.ids[m] : -1;
        id[fm] = (uint32_t)a < (uint32_t)p.adapters ? a : -1;
        rows[fm] = (uint32_t)__builtin_amdgcn_ballot_w64(id[fm] >= 0);
        any |= rows[fm];
    }
    if (any == 0)
        return;
    const int h = lane >> 5;
    const uint32_t bytes = (uint32_t)p.N * (uint32_t)p.up_ld * 2u;   // below 2^31 (host)
    const uint32_t voff = (uint32_t)(c0 + (lane & 31)) * (uint32_t)p.up_ld * 2u + (uint32_t)(8 * h) * 2u;
    auto load_up = [&](int a, int fn, int rs) {
        return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                             make_rsrc(p.up + (int64_t)a * p.up_stride, bytes),
                                             rs + 8 * h < p.rank && c0 + fn * 32 + (lane & 31) < p.N
                                                 ? voff + (uint32_t)(fn * 32) * (uint32_t)p.up_ld * 2u
                                                 : kOutOfRange,
                                             (uint32_t)rs * 2u, 0));
    };
    // the walk: the adapter of the first row left, until none is; this split's share
    uint32_t left[FM];
    int nth = 0;
    auto start = [&] {
#pragma unroll
        for (int fm = 0; fm < FM; ++fm)
            left[fm] = rows[fm];
        nth = 0;
    };
    auto next = [&]() -> int {
        for (;;) {
            int a = -1;
#pragma unroll
            for (int fm = 0; fm < FM; ++fm)
                if (a < 0 && left[fm])
                    a = __builtin_amdgcn_readlane(id[fm], __builtin_ctz(left[fm]));
            if (a < 0)
                return -1;
#pragma unroll
            for (int fm = 0; fm < FM; ++fm)
                left[fm] &= ~(uint32_t)__builtin_amdgcn_ballot_w64(id[fm] == a);
            const bool mine = nth % p.splits == split;
            ++nth;
            if (mine)
                return a;
        }
    };
    // the next NB adapters and their fragments of ranks rs .. +16
    int a[NB];
    u32x4 up[NB][FN];
    auto fetch = [&](int rs) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            a[b] = b == 0 || a[b - 1] >= 0 ? next() : -1;
            if (a[b] >= 0)
#pragma unroll
                for (int fn = 0; fn < FN; ++fn)
                    up[b][fn] = load_up(a[b], fn, rs);
        }
    };
    // the wave's low-rank values of ranks rs + 8 h .. +8 (the first split's, to begin with)
    f32x4 low[FM][2];
    auto fetch_low = [&](int rs) {
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) {
            low[fm][0] = low[fm][1] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
            if (id[fm] >= 0 && rs + 8 * h < p.rank) {
                const int m = r0 + fm * 32 + (lane & 31);
                const float *src = p.low + (int64_t)m * p.rank_pad + rs + 8 * h;
                low[fm][0] = *reinterpret_cast<const f32x4 *>(src);
                low[fm][1] = *reinterpret_cast<const f32x4 *>(src + 4);
            }
        }
    };
    float scale[FM];                   // (times the row's units)
    bool units = false;                // some row's are not 1
    auto shift_of = [&](int fm) {      // the units' exponent, without a register of its own
        return id[fm] >= 0 ? __builtin_amdgcn_frexp_expf(scale[fm]) - __builtin_amdgcn_frexp_expf(p.scale[id[fm]]) : 0;
    };
    auto rescale = [&](int fm, int by) {
        const float f = __builtin_ldexpf(1.0f, by);
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc[fn][fm][e] *= f;
    };
    start();
    fetch(0);
    if constexpr (AHEAD)
        fetch_low(0);
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
        scale[fm] = id[fm] >= 0 ? p.scale[id[fm]] : 0.0f;
    for (int rs = 0; rs < p.rank; rs += 16) {
        if constexpr (!AHEAD)
            fetch_low(rs);
        // scaled, and split in parts
        u32x4 part[NP][FM];
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) {
            f32x4 v0 = low[fm][0], v1 = low[fm][1];
            if (p.low_splits > 1 && id[fm] >= 0 && rs + 8 * h < p.rank) {
                const int m = r0 + fm * 32 + (lane & 31);
                const float *src = p.low + (int64_t)m * p.rank_pad + rs + 8 * h;
                for (int s = 1; s < p.low_splits; ++s) {
                    src += p.low_stride;
                    v0 += *reinterpret_cast<const f32x4 *>(src);
                    v1 += *reinterpret_cast<const f32x4 *>(src + 4);
                }
            }
            v0 *= scale[fm];
            v1 *= scale[fm];
            if constexpr (IN == IN_FP16) {
                float top = 0.0f;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    top = fmaxf(top, fmaxf(__builtin_fabsf(v0[d]), __builtin_fabsf(v1[d])));
                const unsigned bits = __builtin_bit_cast(unsigned, top);
                const auto both = __builtin_amdgcn_permlane32_swap(bits, bits, false, false);
                const unsigned lower = both[0], upper = both[1];   // (a row's 16 ranks are in two lanes)
                top = fmaxf(__builtin_bit_cast(float, lower), __builtin_bit_cast(float, upper));
                const bool out = top > 0.0f && __builtin_isfinite(top) && (top < 0.125f || top >= 32768.0f);
                if (__builtin_amdgcn_ballot_w64(out)) {
                    mfma_settle();
                    // top in [2^(e - 1), 2^e): to just below 2^15; but units that a large
                    // value has lowered are not raised again, over what it left in the sums
                    const int e = __builtin_amdgcn_frexp_expf(top), was = shift_of(fm);
                    const int to = max(-60, min(60, was + 15 - e));
                    const int by = out && (to < was || was >= 0) ? to - was : 0;
                    rescale(fm, by);
                    scale[fm] = __builtin_ldexpf(scale[fm], by);
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        v0[d] = __builtin_ldexpf(v0[d], by);
                        v1[d] = __builtin_ldexpf(v1[d], by);
                    }
                    units = true;
                }
            }
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                uint16_t a[NP], b[NP];
                split16<IN>(d < 2 ? v0[2 * d] : v1[2 * d - 4], a);
                split16<IN>(d < 2 ? v0[2 * d + 1] : v1[2 * d - 3], b);
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    part[i][fm][d] = (uint32_t)a[i] | (uint32_t)b[i] << 16;
            }
        }
        // (the next ranks' values are on their way while these are multiplied)
        if (AHEAD && rs + 16 < p.rank)
            fetch_low(rs + 16);
        const u32x4 zero = {0u, 0u, 0u, 0u};
        bool apart = false;
        for (;;) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if (a[b] < 0)
                    continue;
                uint32_t special = 0;
#pragma unroll
                for (int fn = 0; fn < FN; ++fn)
                    special |= has_special<IN>(up[b][fn]);
                if (__builtin_amdgcn_ballot_w64(special != 0)) {
                    apart = true;
                    continue;
                }
#pragma unroll
                for (int fm = 0; fm < FM; ++fm) {
                    const bool own = id[fm] == a[b];
                    if (__builtin_amdgcn_ballot_w64(own) == 0)
                        continue;
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        const u32x4 t = own ? part[i][fm] : zero;
#pragma unroll
                        for (int fn = 0; fn < FN; ++fn)
                            acc[fn][fm] = mfma32x32x16<IN>(up[b][fn], t, acc[fn][fm]);
                    }
                }
            }
            if (a[NB - 1] < 0)
                break;
            fetch(rs);
        }
        if (apart) {
            // the adapters left out above, one at a time
            start();
            for (int s = next(); s >= 0; s = next()) {
                uint32_t special = 0;
#pragma unroll
                for (int fn = 0; fn < FN; ++fn)
                    special |= has_special<IN>(load_up(s, fn, rs));
                if (__builtin_amdgcn_ballot_w64(special != 0) == 0)
                    continue;
#pragma unroll
                for (int fm = 0; fm < FM; ++fm) {
                    const bool own = id[fm] == s;
                    if (__builtin_amdgcn_ballot_w64(own) == 0)
                        continue;
#pragma unroll
                    for (int fn = 0; fn < FN; ++fn) {
                        int again = s;                    // (a load of its own: registers)
                        asm volatile("" : "+s"(again));
                        add_special<IN>(
                            load_up(again, fn, rs), own ? part[0][fm] : zero, own,
                            [&](u32x4 x) {
#pragma unroll
                                for (int i = 0; i < NP; ++i)
                                    acc[fn][fm] = mfma32x32x16<IN>(x, own ? part[i][fm] : zero, acc[fn][fm]);
                            },
                            [&](u32x4 x, u32x4 y) { acc[fn][fm] = mfma32x32x16<IN_BF16>(x, y, acc[fn][fm]); });
                    }
                }
            }
        }
        if (rs + 16 < p.rank) {
            start();
            fetch(rs + 16);
        }
    }
    mfma_settle();
    if (units)
#pragma unroll
        for (int fm = 0; fm < FM; ++fm)
            rescale(fm, -shift_of(fm));
}

}  // namespace gnt
