// layer_common.hpp -- pieces shared by the kernels of a feed-forward layer's products:
// argument blocks, activations with their slopes, and what the tiles do with their sums.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../gemm_nt_common.hpp"

namespace gnt {

enum : int { GATE_RELU = 1, GATE_GELU = 2, GATE_SILU = 3 };

// Words that a launch sets to zero.
struct ClearList {
    unsigned *at[4];
    int count[4];
};

__device__ __forceinline__ void clear_list(const ClearList &l, int id, int threads)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        for (int j = id; j < l.count[i]; j += threads)
            l.at[i][j] = 0u;
}

// The gated block's products.  B and B2 are the gate's and the up projection's weights,
// `cols` rows each, in turn groups of eight (GNT_EXT_PAIRED): N, or the contraction of the
// input gradient, counts both, 2 cols rounded up to whole groups.
struct PairedArgs : KernelArgs {
    const uint16_t *B2;
    int ldb2;
    int cols;
    const uint16_t *dh;         // backward: the block's output gradient [M][cols]
    int lddh;
    // FP16 backward, what the units of rows and columns are made of (gate_units): the finite |dh|'s
    // largest bits of each row [M] and of each chunk of rows' columns [col_chunks][col_step], and
    // kNormParts partial maxima of the squared norms of X's rows and of the weights' rows; and the
    // units' reciprocals [M] and [cols], which the sums' gradients leave for the products over
    // them (null: no units)
    const uint16_t *row_most;
    const uint16_t *col_most;
    int col_chunks, col_step;
    const float *norms;
    float *row_back, *col_back;
    void *C2;                   // weight gradients: C is the gate's, C2 the up projection's; FP16
                                // gradients of the sums: C in its rows' units (or null), C2 its columns'
    ClearList clear;            // gradients of the sums: cleared on the way
};

constexpr int kNormParts = 512;

// An opaque copy of the lane id: what an epilogue derives from it is computed there, and
// not held across the main loop, whose registers are all taken.
__device__ __forceinline__ int fresh_lane(int lane)
{
    asm volatile("" : "+v"(lane));
    return lane;
}

__device__ __forceinline__ float from_bits16(int in, uint32_t h)
{
    return in == IN_BF16 ? __builtin_bit_cast(float, h << 16)
                         : static_cast<float>(__builtin_bit_cast(_Float16, (uint16_t)h));
}

// Phi(x) and phi(x), the normal distribution and its density.  Phi(-|x|) = exp(-x^2 / 2)
// t q(t), t = 1 / (1 + 0.3 |x|): erfcx(|x| / sqrt 2) / 2 is smooth in t, and q is its quotient by
// t as a polynomial fitted here (Chebyshev nodes on 0 <= |x| <= 14.5, relative error
// made even by reweighting): 1.7e-7 of Phi, 5e-7 evaluated in FP32.  So the tail keeps its
// relative accuracy, and the slope takes the same exponential.
__device__ __forceinline__ void normal_cdf(float x, float &cdf, float &pdf)
{
    const float a = fabsf(x);
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.3f * a);
    float q = 0.0354238897562027f;
    q = q * t - 0.15615904331207275f;
    q = q * t + 0.20455773174762726f;
    q = q * t - 0.05203482508659363f;
    q = q * t + 0.12769216299057007f;
    q = q * t + 0.10017584264278412f;
    q = q * t + 0.12071215361356735f;
    q = q * t + 0.11963200569152832f;
    const float e = __expf(-0.5f * x * x);
    const float low = e * (t * q);
    cdf = x < 0.0f ? low : 1.0f - low;
    pdf = 0.39894228040143268f * e;
}

// act(v); with `slope` also act'(v) (0 at ReLU's corner).  A NaN stays one.
template <bool SLOPE>
__device__ __forceinline__ float gate_value(int act, float v, float &slope)
{
    if (act == GATE_SILU) {
        const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-v));
        if constexpr (SLOPE)
            slope = s + v * s * (1.0f - s);
        return v * s;
    }
    if (act == GATE_GELU) {
        float cdf, pdf;
        normal_cdf(v, cdf, pdf);
        if constexpr (SLOPE)
            slope = cdf + v * pdf;
        return v * cdf;
    }
    if constexpr (SLOPE)
        slope = v <= 0.0f ? 0.0f : v > 0.0f ? 1.0f : v;
    return v <= 0.0f ? 0.0f : v;
}

template <int OUT>
__device__ __forceinline__ uint32_t to_bits16(float x)
{
    if constexpr (OUT == OUT_BF16)
        return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
    else
        return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
}

// 16 bytes of values at the alignment of one: the memory unit takes them at any address, so rows
// of odd lengths need no other path (with one of single values for them, the gated block of 1500
// rows and 5461 FP16 columns 143 us, 130 with this; quantizing 4000 x 4095 BF16 29 and 16, FP32
// 38 and 16).
typedef uint32_t run16_t __attribute__((ext_vector_type(4), aligned(2)));
typedef float run32_t __attribute__((ext_vector_type(4), aligned(4)));

// `count` (1 .. 8, or 4 of FP32) consecutive values of a row at C, element index idx: one
// 16-byte store where all are there, of 16-bit values with the non-temporal policy where
// NT (results; what the next launch reads stays in the caches).
template <int OUT, int V, bool NT = true>
__device__ __forceinline__ void store_run(void *C, int64_t idx, const float (&x)[V], int count)
{
    if constexpr (OUT == OUT_FP32) {
        float *c = static_cast<float *>(C) + idx;
        if (count >= V) {
#pragma unroll
            for (int i = 0; i < V; i += 4)
                *reinterpret_cast<run32_t *>(c + i) = (run32_t){x[i], x[i + 1], x[i + 2], x[i + 3]};
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < count)
                    c[i] = x[i];
        }
    } else {
        static_assert(V == 8, "16 bytes");
        uint16_t *c = static_cast<uint16_t *>(C) + idx;
        run16_t w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = to_bits16<OUT>(x[2 * i]) | to_bits16<OUT>(x[2 * i + 1]) << 16;
        if (count >= V) {
            if constexpr (NT)
                __builtin_nontemporal_store(w, reinterpret_cast<run16_t *>(c));
            else
                *reinterpret_cast<run16_t *>(c) = w;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < count)
                    c[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        }
    }
}

// The gated block's output: act(gate) * up of a wave's accumulators (gate and up in one
// lane, registers 8 u + e and 8 u + 4 + e) into C [M][cols], whose columns are half the
// tile's.  The wave's block is staged as FP32 rows of 16 FN values in its own LDS, chunk c of
// row r at c ^ (r mod the chunks), and read back as 16-byte pieces of rows.
template <int OUT, int FN, int FM>
__device__ __forceinline__ void store_gated(const PairedArgs &p, const f32x16 (&acc)[FN][FM], int r0, int c0,
                                            uint8_t *stage, int lane_id)
{
    const int lane = fresh_lane(lane_id);
    constexpr int CPR = 4 * FN, ROWB = 16 * CPR, KEYM = CPR - 1;
    const int h = lane >> 5;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = fm * 32 + (lane & 31), c = 4 * fn + 2 * u + h;
                f32x4 y;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float slope;
                    y[e] = gate_value<false>(p.act, acc[fn][fm][8 * u + e], slope) * acc[fn][fm][8 * u + 4 + e];
                }
                *reinterpret_cast<f32x4 *>(stage + r * ROWB + ((c ^ (r & KEYM)) * 16)) = y;
            }
    wait_lgkmcnt0();
    constexpr int V = OUT == OUT_FP32 ? 4 : 8;        // values per lane
    constexpr int LPR = 16 * FN / V, RPS = 64 / LPR;  // lanes per row, rows per step
#pragma unroll
    for (int j = 0; j < 32 * FM / RPS; ++j) {
        const int r = j * RPS + lane / LPR, c = (lane % LPR) * (V / 4);
        const int m = r0 + r, n = c0 / 2 + 4 * c;
        float y[V];
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(stage + r * ROWB + (((c + i) ^ (r & KEYM)) * 16));
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[4 * i + e] = v[e];
        }
        if (m < p.M && n < p.cols)
            store_run<OUT, V>(p.C, (int64_t)m * p.ldc + n, y, p.cols - n);
    }
}

// FP16 gradients of the pre-activations, in units.  |dg| = |dh u act'(g)| and |du| = |dh act(g)| are
// at most |dh| B, B = 1.13 max ||x_m|| max ||w_f|| (Cauchy and Schwarz; act' is at most 1.129, and
// |act(g)| at most |g|).  So an exponent of 13 - floor(log2 max|dh|) - floor(log2 B) keeps them below
// 2^15 whatever they are, of each row with its own max|dh| for dx and of each column with its
// own for the weights' gradients, as the sums that they enter are apart in the same way: neither a
// large sum nor a large row or entry of dh takes bits from the rest.  B is above typical sums of
// K products by sqrt(K) / 3 or so, 4 of the 29 binades that have all their bits.
__device__ __forceinline__ int bound_exponent(const float *norms, int lane)
{
    float x = 0.0f, w = 0.0f;
#pragma unroll
    for (int j = 0; j < kNormParts; j += 256) {
        const f32x4 px = *reinterpret_cast<const f32x4 *>(norms + j + 4 * lane);
        const f32x4 pw = *reinterpret_cast<const f32x4 *>(norms + kNormParts + j + 4 * lane);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x = fmaxf(x, px[i]), w = fmaxf(w, pw[i]);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        x = fmaxf(x, __shfl_xor(x, o));
        w = fmaxf(w, __shfl_xor(w, o));
    }
    // (1.13^2 and 2% for the norms' own roundings; of 2^-96 .. 2^109, or 0)
    const uint32_t b = __builtin_amdgcn_readfirstlane(__builtin_bit_cast(uint32_t, 1.3f * x * w));
    return b == 0 ? 0 : ((int)(b >> 23) - 127) >> 1;
}

// The unit's exponent of what has the largest bits `most` (FP16, finite): -57 .. 86.
__device__ __forceinline__ int unit_exponent(uint32_t most, int bound)
{
    if (most == 0)
        return 0;
    const int log2 = most >= 0x400u ? (int)(most >> 10) - 15 : 7 - __builtin_clz(most);
    return 13 - log2 - bound;
}

__device__ __forceinline__ uint32_t column_most(const PairedArgs &p, int f)
{
    uint32_t b = 0;
    for (int c = 0; c < p.col_chunks; c += 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)                  // (all of them at once; past the last, that one again)
            b = max(b, (uint32_t)p.col_most[(int64_t)min(c + i, p.col_chunks - 1) * p.col_step + f]);
    }
    return b;
}

// The gradients of the pre-activations from their sums, dg = dh u act'(g) and du = dh act(g),
// into C [M][N] in the sums' own layout (N = 2 cols rounded up, rows 16-byte aligned).  The
// wave's part of dh, 16 FN columns of 32 rows a pass, comes through its LDS in 16-byte
// pieces of rows (read in the accumulators' layout a load would touch 32 rows for 8 bytes
// each), and the results leave the same way.  Columns at or past `cols` (the last group's
// rest) get zeros.  FP16: once in units of the row, once of the column, of at most two fn's columns a
// pass (as both results of four would not fit the 16 KB that a wave of the ping-pong tile has).
template <int IN, int FN, int FM>
__device__ __forceinline__ void store_gate_gradients(const PairedArgs &p, const f32x16 (&acc)[FN][FM], int r0,
                                                     int c0, uint8_t *stage, int lane_id)
{
    constexpr bool UNITS = IN == IN_FP16;
    constexpr int PN = UNITS && FN > 2 ? 2 : FN;                                     // fn a pass
    constexpr int CPR = 2 * PN, ROWB = 16 * CPR, KEYM = CPR - 1, RPS = 64 / CPR;     // dh
    constexpr int CPO = 4 * PN, ROWO = 16 * CPO, KEYO = CPO - 1, RPO = 64 / CPO;     // results
    static_assert(32 * (ROWB + (UNITS ? 2 : 1) * ROWO) + (UNITS ? 64 * FN : 0) <= (FN > 1 ? 16384 : 8192),
                  "the least that a wave has: of the ping-pong tile, and of the two-stage ring");
    const int lane = fresh_lane(lane_id);
    const int h = lane >> 5;
    uint8_t *out = stage + 32 * ROWB, *out2 = out + 32 * ROWO;
    float *columns = reinterpret_cast<float *>(out2 + 32 * ROWO);      // their units
    clear_list(p.clear, blockIdx.x * blockDim.x + threadIdx.x, gridDim.x * blockDim.x);
    int rows[FM];
    if constexpr (UNITS) {
        const int f = c0 / 2 + lane;
        const uint32_t most = column_most(p, min(f, p.cols - 1));
        uint32_t mosts[FM];
#pragma unroll
        for (int fm = 0; fm < FM; ++fm)
            mosts[fm] = p.row_most[min(r0 + fm * 32 + (lane & 31), p.M - 1)];
        const int bound = bound_exponent(p.norms, lane), column = unit_exponent(most, bound);
        if (lane < 16 * FN) {
            columns[lane] = __builtin_ldexpf(1.0f, column);
            if (r0 == 0 && f < p.cols)
                p.col_back[f] = __builtin_ldexpf(1.0f, -column);
        }
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) {
            rows[fm] = unit_exponent(mosts[fm], bound);
            const int m = r0 + fm * 32 + lane;
            if (c0 == 0 && lane < 32 && m < p.M)
                p.row_back[m] = __builtin_ldexpf(1.0f, -rows[fm]);
        }
    }
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
        const int r = lane & 31;
        float row = 1.0f;
        if constexpr (UNITS)
            row = __builtin_ldexpf(1.0f, rows[fm]);
#pragma unroll
        for (int f1 = 0; f1 < FN; f1 += PN) {
            const int f0 = c0 / 2 + 16 * f1;
#pragma unroll
            for (int j = 0; j < 32 / RPS; ++j) {
                const int rd = j * RPS + lane / CPR, c = lane % CPR;
                const int m = r0 + fm * 32 + rd, n = f0 + 8 * c;
                u32x4 w = {0u, 0u, 0u, 0u};
                if (m < p.M && n < p.cols) {
                    const uint16_t *src = p.dh + (int64_t)m * p.lddh + n;
                    if (n + 8 <= p.cols) {
                        w = *reinterpret_cast<const run16_t *>(src);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (n + i < p.cols)
                                w[i >> 1] |= (uint32_t)src[i] << (16 * (i & 1));
                    }
                }
                *reinterpret_cast<u32x4 *>(stage + rd * ROWB + ((c ^ (rd & KEYM)) * 16)) = w;
            }
            wait_lgkmcnt0();
#pragma unroll
            for (int fn = 0; fn < PN; ++fn)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int ch = 2 * fn + u, n = f0 + 8 * ch + 4 * h;
                    const f32x16 &sums = acc[f1 + fn][fm];
                    const u32x2 w = *reinterpret_cast<const u32x2 *>(stage + r * ROWB + ((ch ^ (r & KEYM)) * 16) + 8 * h);
                    float dg[4], du[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float d = from_bits16(IN, (w[e >> 1] >> (16 * (e & 1))) & 0xffffu);
                        float slope;
                        const float a = gate_value<true>(p.act, sums[8 * u + e], slope);
                        const bool in = n + e < p.cols;
                        dg[e] = in ? d * sums[8 * u + 4 + e] * slope : 0.0f;
                        du[e] = in ? d * a : 0.0f;
                    }
                    // column 32 fn + 16 u + 4 h of dg and, eight on, of du
                    auto put = [&](uint8_t *to, f32x4 unit) {
                        uint32_t b[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            b[e] = to_bits16<IN>(unit[e] * dg[e]), b[4 + e] = to_bits16<IN>(unit[e] * du[e]);
                        uint8_t *at = to + r * ROWO + 8 * h;
                        *reinterpret_cast<u32x2 *>(at + (((2 * ch) ^ (r & KEYO)) * 16)) = (u32x2){b[0] | b[1] << 16, b[2] | b[3] << 16};
                        *reinterpret_cast<u32x2 *>(at + (((2 * ch + 1) ^ (r & KEYO)) * 16)) = (u32x2){b[4] | b[5] << 16, b[6] | b[7] << 16};
                    };
                    put(out, (f32x4){row, row, row, row});
                    if constexpr (UNITS)
                        put(out2, *reinterpret_cast<const f32x4 *>(columns + 16 * f1 + 8 * ch + 4 * h));
                }
            wait_lgkmcnt0();
#pragma unroll
            for (int j = 0; j < 32 / RPO; ++j) {
                const int ro = j * RPO + lane / CPO, c = lane % CPO;
                const int m = r0 + fm * 32 + ro, n = c0 + 32 * f1 + 8 * c;
                const int at = ro * ROWO + ((c ^ (ro & KEYO)) * 16);
                const bool in = m < p.M && n < p.N;
                if (in && (!UNITS || p.C))
                    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p.C) + (int64_t)m * p.ldc + n) =
                        *reinterpret_cast<const u32x4 *>(out + at);
                if constexpr (UNITS)
                    if (in && p.C2)
                        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p.C2) + (int64_t)m * p.ldc + n) =
                            *reinterpret_cast<const u32x4 *>(out2 + at);
            }
            wait_lgkmcnt0();
        }
    }
}

// Takes FP16 gradients' units back out of sums over them: of each of X's rows, or (COLS, weight
// gradients) of each column of theirs, tile row R the one that store_paired_rows says.
template <int IN, bool COLS, int FN, int FM>
__device__ __forceinline__ void unscale(const PairedArgs &p, f32x16 (&acc)[FN][FM], int r0, int lane_id)
{
    if constexpr (IN == IN_FP16) {
        const float *back = COLS ? p.col_back : p.row_back;
        if (!back)                                   // (sums over nothing)
            return;
        const int lane = fresh_lane(lane_id);
        float f[FM];
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) {
            const int r = r0 + fm * 32 + (lane & 31);
            f[fm] = back[COLS ? min((r >> 4) * 8 + (r & 7), p.cols - 1) : min(r, p.M - 1)];
        }
#pragma unroll
        for (int fm = 0; fm < FM; ++fm)
#pragma unroll
            for (int fn = 0; fn < FN; ++fn)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    acc[fn][fm][e] *= f[fm];
    }
}

// The weight gradients' store: tile row R is row 8 (R / 16) + R mod 8 of the gate's array
// (C) or the up projection's (C2), by R / 8 mod 2.  Staged as FP32, 32 rows a pass, and
// read back as 16-byte pieces of rows.
template <int OUT, int FN, int FM>
__device__ __forceinline__ void store_paired_rows(const PairedArgs &p, const f32x16 (&acc)[FN][FM], int r0, int c0,
                                                  uint8_t *stage, int lane_id)
{
    const int lane = fresh_lane(lane_id);
    constexpr int CPR = 8 * FN, ROWB = 16 * CPR, KEYM = CPR < 16 ? CPR - 1 : 15;
    constexpr int V = OUT == OUT_FP32 ? 4 : 8;
    constexpr int LPR = 32 * FN / V, RPS = 64 / LPR;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = lane & 31, c = 8 * fn + 2 * q + (lane >> 5);
                const f32x4 v = {acc[fn][fm][4 * q], acc[fn][fm][4 * q + 1], acc[fn][fm][4 * q + 2],
                                 acc[fn][fm][4 * q + 3]};
                *reinterpret_cast<f32x4 *>(stage + r * ROWB + ((c ^ (r & KEYM)) * 16)) = v;
            }
        wait_lgkmcnt0();
#pragma unroll
        for (int j = 0; j < 32 / RPS; ++j) {
            const int r = j * RPS + lane / LPR, c = (lane % LPR) * (V / 4);
            const int R = r0 + fm * 32 + r, f = (R >> 4) * 8 + (R & 7), n = c0 + 4 * c;
            float y[V];
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                const f32x4 v = *reinterpret_cast<const f32x4 *>(stage + r * ROWB + (((c + i) ^ (r & KEYM)) * 16));
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[4 * i + e] = v[e];
            }
            if (f < p.cols && n < p.N)
                store_run<OUT, V>((R >> 3) & 1 ? p.C2 : p.C, (int64_t)f * p.ldc + n, y, p.N - n);
        }
        wait_lgkmcnt0();
    }
}

// The product in 8-bit integers: a scale for each row of A and each row of B (or one for
// all: step 0).
struct Int8Args : KernelArgs {
    const float *sa;
    const float *sb;
    int sa_step, sb_step;
};

// Whole INT32 sums to FP32 ones in the values' units: (sum * s_m) * t_n, one rounding of the
// sum (2^-24 of it) and one of each product, in this order so that a sum of zero stays
// zero whatever the scales' product.  Never a K split's: its partials stay integers, so that the
// result is the same whatever the splits, and finite where only a part of the sum is not.  (What
// `whole` is not comes through as it is: a branch round the scales cost the ping-pong tile 2% where
// it came before a reduction, and after one 144 registers in memory.)
template <int FN, int FM>
__device__ __forceinline__ void int8_scale(const Int8Args &p, f32x16 (&acc)[FN][FM], int r0, int c0, int lane_id,
                                           bool whole)
{
    const int lane = fresh_lane(lane_id);
    float s[FM];
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
        s[fm] = p.sa[(int64_t)min(r0 + fm * 32 + (lane & 31), p.M - 1) * p.sa_step];
#pragma unroll
    for (int fn = 0; fn < FN; ++fn)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int n = c0 + fn * 32 + 8 * q + 4 * (lane >> 5);
            float t[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                t[e] = p.sb[(int64_t)min(n + e, p.N - 1) * p.sb_step];
#pragma unroll
            for (int fm = 0; fm < FM; ++fm)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float sum = acc[fn][fm][4 * q + e];
                    acc[fn][fm][4 * q + e] =
                        whole ? (static_cast<float>(__builtin_bit_cast(int, sum)) * s[fm]) * t[e] : sum;
                }
            __builtin_amdgcn_sched_barrier(0);
        }
}

}  // namespace gnt
