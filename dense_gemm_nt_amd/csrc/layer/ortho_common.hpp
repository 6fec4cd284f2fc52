// ortho_common.hpp -- the tiles' part in the orthogonalized update (layer_ortho.hip).
#pragma once

#include "layer_common.hpp"

namespace gnt {

// What a product's sums become (all arrays of a step have rows of a multiple of 8 values, zeros
// past the matrix):
//   SQUARE  t (X X^T - sigma I), FP16
//   POLY    t (b' A + c A^2) from A, FP16
//   STEP    a' X + B X: X in FP32 again, and s X in FP16; in the last step the update
enum : int { ORTHO_SQUARE = 0, ORTHO_POLY = 1, ORTHO_STEP = 2 };

struct OrthoArgs : KernelArgs {
    int mode;
    int all_splits;                    // K splits (p.splits is 1 once they are summed)
    int64_t a_step, b_step, c_step;    // elements between a stack's matrices (16-bit ones)
    const uint16_t *old;               // POLY: A (c_step apart)
    float shift;                       // SQUARE: t sigma
    float scale;                       // STEP: s
    float *x;                          // STEP: X in FP32 (c_step apart, rows of ldc)
    void *update;                      // the last STEP's result (else null), rows of ldu
    int64_t update_step;
    int update_dtype, ldu;
    int update_rows, update_cols;      // of X's shape; `flip`: stored transposed
    int flip, update16;                // update16: its rows allow 16-byte stores
};

// The stack's matrix that a block is of.  (Computed again in the epilogue from the block id,
// as is what follows from it: held across the main loop it would not fit the scalar registers.)
__device__ __forceinline__ int ortho_matrix(const OrthoArgs &p)
{
    return blockIdx.x / (p.tiles_m * p.tiles_n * p.splits);
}

// Block id -> its matrix (p.A and p.B move there), and the tile and split in it.
__device__ __forceinline__ void ortho_map(OrthoArgs &p, int &tm, int &tn, int &split)
{
    const int per = p.tiles_m * p.tiles_n * p.splits;
    const int b = ortho_matrix(p), v = blockIdx.x - b * per;
    p.A += b * p.a_step;
    p.B += b * p.b_step;
    if (p.inreduce)
        map_block_split_minor(v, per, p.tiles_m, p.tiles_n, p.group_m, p.splits, tm, tn, split);
    else
        map_block(v, per, p.tiles_m, p.tiles_n, p.group_m, tm, tn, split);
}

// (before a reduction in the kernel sets p.splits to 1)
__device__ __forceinline__ int ortho_tile(const OrthoArgs &p, int tm, int tn)
{
    return (ortho_matrix(p) * p.tiles_m + tm) * p.tiles_n + tn;
}

__device__ __forceinline__ void store_update(const OrthoArgs &p, int64_t idx, const float (&y)[8], int count)
{
    if (p.update_dtype == OUT_FP32)
        store_run<OUT_FP32, 8>(p.update, idx, y, p.update16 != 0, count);
    else if (p.update_dtype == OUT_FP16)
        store_run<OUT_FP16, 8>(p.update, idx, y, p.update16 != 0, count);
    else
        store_run<OUT_BF16, 8>(p.update, idx, y, p.update16 != 0, count);
}

// A wave's sums, 32 rows a pass through its LDS as FP32 (chunk c of row r at c ^ (r mod
// 16)), read back as eight consecutive values of a row, or for a transposed update of a
// column.
template <int FN, int FM>
__device__ __forceinline__ void store_ortho(const OrthoArgs &p, const f32x16 (&acc)[FN][FM], int r0, int c0,
                                            uint8_t *stage, int lane_id)
{
    constexpr int CPR = 8 * FN, ROWB = 16 * CPR, KEYM = CPR < 16 ? CPR - 1 : 15;
    constexpr int LPR = 4 * FN, RPS = 64 / LPR;
    const int lane = fresh_lane(lane_id);
    const int64_t b = blockIdx.x / (p.tiles_m * p.tiles_n * p.all_splits);
    uint16_t *C = static_cast<uint16_t *>(p.C) + b * p.c_step;
    const uint16_t *old = p.old + b * p.c_step;
    float *x = p.x + b * p.c_step;
    const bool turn = p.mode == ORTHO_STEP && p.update && p.flip;
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
#pragma unroll 2
        for (int j = 0; j < 32 / RPS; ++j) {
            const int r = j * RPS + lane / LPR, c = (lane % LPR) * 2;
            const int m = r0 + fm * 32 + r, n = c0 + 4 * c;
            const int64_t idx = (int64_t)m * p.ldc + n;
            uint8_t *at0 = stage + r * ROWB + ((c ^ (r & KEYM)) * 16), *at1 = stage + r * ROWB + (((c + 1) ^ (r & KEYM)) * 16);
            const f32x4 lo = *reinterpret_cast<const f32x4 *>(at0), hi = *reinterpret_cast<const f32x4 *>(at1);
            float y[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            if (m < p.M && n < p.N) {
                if (p.mode == ORTHO_SQUARE) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[i] = p.alpha * y[i] - (m == n + i ? p.shift : 0.0f);
                    store_run<OUT_FP16, 8>(C, idx, y, true, 8);
                } else if (p.mode == ORTHO_POLY) {
                    const u32x4 w = *reinterpret_cast<const u32x4 *>(old + idx);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[i] = p.alpha * y[i] + p.beta * from_bits16(IN_FP16, (w[i >> 1] >> (16 * (i & 1))) & 0xffffu);
                    store_run<OUT_FP16, 8>(C, idx, y, true, 8);
                } else {
                    const f32x4 xl = *reinterpret_cast<const f32x4 *>(x + idx), xr = *reinterpret_cast<const f32x4 *>(x + idx + 4);
                    float s[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        y[i] = p.alpha * y[i] + p.beta * (i < 4 ? xl[i] : xr[i - 4]);
                        s[i] = p.scale * y[i];
                    }
                    if (!p.update) {
                        *reinterpret_cast<f32x4 *>(x + idx) = (f32x4){y[0], y[1], y[2], y[3]};
                        *reinterpret_cast<f32x4 *>(x + idx + 4) = (f32x4){y[4], y[5], y[6], y[7]};
                        store_run<OUT_FP16, 8>(C, idx, s, true, 8);
                    } else if (turn) {
                        *reinterpret_cast<f32x4 *>(at0) = (f32x4){y[0], y[1], y[2], y[3]};
                        *reinterpret_cast<f32x4 *>(at1) = (f32x4){y[4], y[5], y[6], y[7]};
                    } else if (m < p.update_rows && n < p.update_cols) {
                        store_update(p, b * p.update_step + (int64_t)m * p.ldu + n, y, p.update_cols - n);
                    }
                }
            }
        }
        wait_lgkmcnt0();
        if (turn) {
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
                if (m < p.update_rows && n < p.update_cols)
                    store_update(p, b * p.update_step + (int64_t)n * p.ldu + m, y, p.update_rows - m);
            }
            wait_lgkmcnt0();
        }
    }
}

}  // namespace gnt
