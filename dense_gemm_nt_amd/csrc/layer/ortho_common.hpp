// ortho_common.hpp -- the tiles' part in the orthogonalized update (layer_ortho.hip).
#pragma once

#include "layer_common.hpp"

namespace gnt {

// What a product's sums become (all arrays of a step have rows of a multiple of 8 values, zeros
// past the matrix):
//   SQUARE  t (X X^T - sigma I), FP16
//   POLY    t (b' A + c A^2) from A, FP16
//   STEP    a' X + B X: s X as the sum of two FP16 values, of which the first is what the products
//           take; in the last step the update
// The products' tiles: all but the _MN ones have both operands K-major; _S2 is the 128 x 128
// tile with a two-stage ring, and so two blocks a compute unit.
enum OrthoTile : int { ORTHO_256, ORTHO_256_MN, ORTHO_128, ORTHO_128_S2, ORTHO_128_MN, ORTHO_64, ORTHO_64_MN };

enum : int { ORTHO_SQUARE = 0, ORTHO_POLY = 1, ORTHO_STEP = 2 };

struct OrthoArgs : KernelArgs {
    int mode;
    int all_splits;                    // K splits (p.splits is 1 once they are summed)
    int tiles;                         // of a matrix, of the launch's size or (`quarters`) twice it
    int first;                         // the launch's first tile of the stack's
    int quarters;                      // its tiles are the four quarters of those from `first` on
    int half;                          // tile size of a square of which the lower half is computed
                                       // (0: all of it), each tile below the diagonal stored twice
    int64_t a_step, b_step, c_step;    // elements between a stack's matrices (16-bit ones)
    const uint16_t *old;               // POLY: A (c_step apart)
    float shift;                       // SQUARE: t sigma
    const uint16_t *hi;                // STEP: s X, the first parts, and the second ones, which the
    uint16_t *lo;                      // step replaces (c_step apart, rows of ldc)
    uint16_t *xt;                      // STEP: s X transposed as well (rows of ldt), or null
    int ldt;
    void *update;                      // the last STEP's result (else null), rows of ldu
    int64_t update_step;
    int update_dtype, ldu;
    int update_rows, update_cols;      // of X's shape; `flip`: stored transposed
    int flip;
};

// Tile t of the lower half: tile row tm has tm + 1 of them.
__device__ __forceinline__ void half_order(int t, int &tm, int &tn)
{
    tm = (int)((__builtin_sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    tm += (tm + 1) * (tm + 2) / 2 <= t ? 1 : 0;      // (the root's rounding, either way)
    tm -= tm * (tm + 1) / 2 > t ? 1 : 0;
    tn = t - tm * (tm + 1) / 2;
}

// Block id -> its tile's number in the launch and its split, and the matrix that it is of.  (Computed again in the epilogue, as is what follows
// from it: held across the main loop it would not fit the scalar registers.)
__device__ __forceinline__ int ortho_number(const OrthoArgs &p, int &split)
{
    const int v = xcd_order(blockIdx.x, gridDim.x);
    // (the splits of a tile next to each other: they are summed in the kernel)
    const int t = v / p.all_splits;
    split = v - t * p.all_splits;
    return t;
}

__device__ __forceinline__ int ortho_matrix(const OrthoArgs &p)
{
    int split;
    const int t = ortho_number(p, split);
    return (p.first + (p.quarters ? t >> 2 : t)) / p.tiles;
}

// Block id -> its matrix (p.A and p.B move there), and the tile and split in it; false for a
// quarter past the matrix.
__device__ __forceinline__ bool ortho_map(OrthoArgs &p, int &tm, int &tn, int &split)
{
    const int i = ortho_number(p, split);
    const int g = p.first + (p.quarters ? i >> 2 : i);
    const int b = g / p.tiles, t = g - b * p.tiles;
    p.A += b * p.a_step;
    p.B += b * p.b_step;
    if (p.half)
        half_order(t, tm, tn);
    else
        tile_order(t, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    if (p.quarters) {
        tm = 2 * tm + ((i >> 1) & 1), tn = 2 * tn + (i & 1);
        const int size = p.half >> 1;
        return tm * size < p.M && tn * size < p.N;
    }
    return true;
}

// The tile's number in the launch.
__device__ __forceinline__ int ortho_tile(const OrthoArgs &p)
{
    int split;
    return ortho_number(p, split);
}

__device__ __forceinline__ float half_at(u32x4 w, int i)
{
    return from_bits16(IN_FP16, (w[i >> 1] >> (16 * (i & 1))) & 0xffffu);
}

// x as the sum of two FP16 values: y (the nearest to x) and what it leaves.  22 bits where s x
// is above 2^-3, and 2^-25 absolute below.
__device__ __forceinline__ void two_halves(float (&x)[8], float (&rest)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float h = static_cast<float>(static_cast<_Float16>(x[i]));
        rest[i] = x[i] - h;
        x[i] = h;
    }
}

// Eight consecutive values from element idx of an array of `dtype`, the first `count` of them.
__device__ __forceinline__ void store_values(void *at, int64_t idx, int dtype, const float (&y)[8], int count)
{
    if (dtype == OUT_FP32)
        store_run<OUT_FP32, 8>(at, idx, y, count);
    else if (dtype == OUT_FP16)
        store_run<OUT_FP16, 8>(at, idx, y, count);
    else
        store_run<OUT_BF16, 8>(at, idx, y, count);
}

// A wave's sums, 32 rows a pass through its LDS as FP32 (chunk c of row r at c ^ (r mod
// 16)), read back as eight consecutive values of a row; and, where what is stored is stored
// transposed too (or only so), from there once more as eight of a column.
template <int FN, int FM>
__device__ __forceinline__ void store_ortho(const OrthoArgs &p, const f32x16 (&acc)[FN][FM], int r0, int c0,
                                            uint8_t *stage, int lane_id)
{
    constexpr int CPR = 8 * FN, ROWB = 16 * CPR, KEYM = CPR < 16 ? CPR - 1 : 15;
    constexpr int LPR = 4 * FN, RPS = 64 / LPR;
    const int lane = fresh_lane(lane_id);
    const int64_t b = ortho_matrix(p);
    uint16_t *C = static_cast<uint16_t *>(p.C) + b * p.c_step;
    const uint16_t *old = p.old + b * p.c_step;
    const uint16_t *hi = p.hi + b * p.c_step;
    uint16_t *lo = p.lo + b * p.c_step;
    // where the transposed values go: a square's other half, X's transposed copy, or a tall
    // update
    void *turned = nullptr;
    int ldt = p.ldc, rows_t = p.M, cols_t = p.N, dtype_t = OUT_FP16;
    int64_t base_t = 0;
    if (p.mode != ORTHO_STEP) {
        if (p.half && r0 / p.half != c0 / p.half)
            turned = C;
    } else if (p.update) {
        if (p.flip)
            turned = p.update, base_t = b * p.update_step, ldt = p.ldu, rows_t = p.update_rows, cols_t = p.update_cols,
            dtype_t = p.update_dtype;
    } else if (p.xt) {
        turned = p.xt + b * p.c_step, ldt = p.ldt;
    }
    // steps whose reads from memory go out together, before anything waits for them
    constexpr int STEPS = 32 / RPS, GROUP = STEPS < 4 ? STEPS : 4;
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
#pragma unroll 1
        for (int g = 0; g < STEPS; g += GROUP) {
            u32x4 v[GROUP], w[GROUP];
            auto at = [&](int j, int &m, int &n) {
                m = r0 + fm * 32 + (g + j) * RPS + lane / LPR;
                n = c0 + 8 * (lane % LPR);
                return (int64_t)m * p.ldc + n;
            };
            if (p.mode == ORTHO_STEP) {
#pragma unroll
                for (int j = 0; j < GROUP; ++j) {
                    int m, n;
                    const int64_t idx = at(j, m, n);
                    if (m < p.M && n < p.N) {
                        v[j] = *reinterpret_cast<const u32x4 *>(hi + idx);
                        w[j] = *reinterpret_cast<const u32x4 *>(lo + idx);
                    }
                }
            } else if (p.mode == ORTHO_POLY) {
#pragma unroll
                for (int j = 0; j < GROUP; ++j) {
                    int m, n;
                    const int64_t idx = at(j, m, n);
                    if (m < p.M && n < p.N)
                        w[j] = *reinterpret_cast<const u32x4 *>(old + idx);
                }
            }
#pragma unroll
            for (int j = 0; j < GROUP; ++j) {
                const int r = (g + j) * RPS + lane / LPR, c = (lane % LPR) * 2;
                int m, n;
                const int64_t idx = at(j, m, n);
                uint8_t *at0 = stage + r * ROWB + ((c ^ (r & KEYM)) * 16), *at1 = stage + r * ROWB + (((c + 1) ^ (r & KEYM)) * 16);
                const f32x4 y0 = *reinterpret_cast<const f32x4 *>(at0), y1 = *reinterpret_cast<const f32x4 *>(at1);
                float y[8] = {y0[0], y0[1], y0[2], y0[3], y1[0], y1[1], y1[2], y1[3]};
                if (m >= p.M || n >= p.N)
                    continue;
                if (p.mode == ORTHO_SQUARE) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[i] = p.alpha * y[i] - (m == n + i ? p.shift : 0.0f);
                    store_run<OUT_FP16, 8, false>(C, idx, y, 8);
                } else if (p.mode == ORTHO_POLY) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[i] = p.alpha * y[i] + p.beta * half_at(w[j], i);
                    store_run<OUT_FP16, 8, false>(C, idx, y, 8);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[i] = p.alpha * y[i] + p.beta * (half_at(v[j], i) + half_at(w[j], i));
                    if (!p.update) {
                        float z[8];
                        two_halves(y, z);
                        store_run<OUT_FP16, 8, false>(C, idx, y, 8);
                        store_run<OUT_FP16, 8, false>(lo, idx, z, 8);
                    } else if (!turned && m < p.update_rows && n < p.update_cols) {
                        store_values(p.update, b * p.update_step + (int64_t)m * p.ldu + n, p.update_dtype, y,
                                     p.update_cols - n);
                    }
                }
                if (turned) {
                    *reinterpret_cast<f32x4 *>(at0) = (f32x4){y[0], y[1], y[2], y[3]};
                    *reinterpret_cast<f32x4 *>(at1) = (f32x4){y[4], y[5], y[6], y[7]};
                }
            }
        }
        wait_lgkmcnt0();
        if (turned) {
            // four lanes a column of the block, eight of its 32 rows each
            const int m = r0 + fm * 32 + 8 * (lane & 3);
#pragma unroll 1
            for (int j = 0; j < 2 * FN; ++j) {
                const int c = 16 * j + (lane >> 2), n = c0 + c;
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = 8 * (lane & 3) + i;
                    y[i] = *reinterpret_cast<const float *>(stage + r * ROWB + (((c >> 2) ^ (r & KEYM)) * 16) + (c & 3) * 4);
                }
                if (m < rows_t && n < cols_t)
                    store_values(turned, base_t + (int64_t)n * ldt + m, dtype_t, y, rows_t - m);
            }
            wait_lgkmcnt0();
        }
    }
}

}  // namespace gnt
