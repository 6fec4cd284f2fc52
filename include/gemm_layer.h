/*
 * gemm_layer.h -- C ABI of the MI355X (gfx950) products of a feed-forward layer:
 * the gated block and its gradients, the product in 8-bit integers with a
 * scale for each token and output channel, and the orthogonalized update of a
 * weight.  Built as libgemm_layer.so, beside gemm_nt.h's library, whose types,
 * status codes and epilogue it uses.
 *
 * Storage, types, rounding: row-major with element strides; operands BF16 or
 * FP16 (all of one call's 16-bit operands share the type) or INT8; FP32 or INT32
 * sums; results rounded once to nearest even.  Limits: rows below 2^30, sizes
 * below 2^31, fewer than 2^23 output tiles, leading dimensions of operands
 * below 2^22 and multiples of 8 (INT8: below 2^23, of 16), operand bases
 * 16-byte aligned; outputs, and dH, need their element's alignment.  Outputs
 * and the workspace must not overlap the operands or each other (not checked
 * here; but for U, which may be G).  For given arguments every call on the same
 * device returns the same bits.
 *
 * Workspaces: no handle; a call that needs one takes a device workspace of the
 * caller's, 256-byte aligned and at least as large as the matching *_workspace
 * function says for the same sizes.  Nothing needs to be in it before a call, and
 * nothing is kept in it between calls.  Two calls that may run concurrently
 * (different streams, two graphs' replays) need workspaces of their own.  A
 * call allocates nothing, reads nothing on the host and only enqueues work on
 * `stream`, for the device that is current; it can be captured into a HIP graph.
 *
 * Errors: GEMM_ERR_INVALID_ARG for null pointers, negative sizes, leading
 * dimensions that are too small, unknown modes and a workspace that is too
 * small; GEMM_ERR_UNSUPPORTED for types and sizes outside the limits;
 * GEMM_ERR_MISALIGNED; GEMM_ERR_HIP.  On an error nothing is enqueued, but for
 * GEMM_ERR_HIP, after which part of a call's launches may be.
 */
#ifndef GEMM_LAYER_H
#define GEMM_LAYER_H

#include <stdint.h>

#include "gemm_nt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The gate's activation: max(0, x), x Phi(x) (the exact form), x / (1 + exp(-x)). */
typedef enum { GEMM_GATE_RELU = 1, GEMM_GATE_GELU = 2, GEMM_GATE_SILU = 3 } gemm_gate_t;

/* The gated block: H = act(X Wg^T) * (X Wu^T), X [M][K], Wg and Wu [F][K], H [M][F] of
 * out_dtype (GEMM_BF16, GEMM_FP16, GEMM_FP32).  Both sums, the activation and the product
 * are FP32; H is rounded once.  One kernel makes both sums and H of them, in one launch or, where
 * the tiles' last pass over the machine would be mostly empty, two.  K splits (few tiles) put FP32
 * partials of the sums into the workspace, which the kernel adds up (a launch that clears counters
 * is before it) or a second pass.
 *   K % 8 == 0; F below 2^21.  K = 0: act(0) * 0. */
gemm_status_t gemm_gated_workspace(int64_t M, int64_t F, int64_t K, int64_t *bytes);
gemm_status_t gemm_run_gated(const void *X, const void *Wg, const void *Wu, void *H, int64_t M,
                             int64_t F, int64_t K, int64_t ldx, int64_t ldwg, int64_t ldwu,
                             int64_t ldh, int in_dtype, int out_dtype, int activation,
                             void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* Gradients of H = act(g) * u, g = X Wg^T, u = X Wu^T, for dH [M][F] of the operands'
 * type (any leading dimension >= F):
 *   dg = dH u act'(g), du = dH act(g)
 *   dX = dg Wg + du Wu     [M][K], dx_dtype
 *   dWg = dg^T X, dWu = du^T X     [F][K] contiguous, grad_dtype, written whole
 * Nothing of the forward call is needed: g and u are computed again, in FP32, and so are dg and
 * du, which are then rounded to the operands' type once, relative to the value 2^-9 at most for
 * BF16 and 2^-12 for FP16.  So an FP32 result is no more exact than that.  FP16's are held in units
 * of powers of two, for dX one of each row, for the weights' gradients one of each column of dH:
 * what is below 2^-27 of the largest finite |dH| of the row (column) times B loses bits, and what
 * is below 2^-38 all of them, B = 1.13 max ||X[m]|| max(||Wg[f]||, ||Wu[f]||) over the finite rows, which
 * no factor of dH exceeds.  So no finite gradient ends FP16's range on the way, and an infinity or NaN
 * in dH is in its own row of dX and its own column's dWg and dWu only.
 * dX may be NULL (not computed), and so may dWg and dWu, both or neither.  act' of ReLU
 * is 0 at 0.  M = 0 writes zeros to dWg and dWu, F = 0 to dX. */
gemm_status_t gemm_gated_backward_workspace(int64_t M, int64_t F, int64_t K, int64_t *bytes);
/* (the one above is enough for either type; BF16 operands need about half of it) */
gemm_status_t gemm_gated_backward_workspace_of(int64_t M, int64_t F, int64_t K, int in_dtype,
                                               int64_t *bytes);
gemm_status_t gemm_run_gated_backward(const void *dH, const void *X, const void *Wg,
                                      const void *Wu, void *dX, void *dWg, void *dWu, int64_t M,
                                      int64_t F, int64_t K, int64_t lddh, int64_t ldx,
                                      int64_t ldwg, int64_t ldwu, int64_t lddx, int in_dtype,
                                      int dx_dtype, int grad_dtype, int activation,
                                      void *workspace, int64_t workspace_bytes,
                                      hipStream_t stream);

/* Rows of X [M][K] (GEMM_BF16, GEMM_FP16 or GEMM_FP32; any leading dimension >= K) in 8-bit
 * integers: scale[m] = max |X[m,:]| / 127, codes[m][k] = X[m][k] / scale[m] to the nearest
 * integer, even at a tie, in -127 .. 127; both quotients are FP32 numbers, rounded to
 * nearest.  A row of zeros has scale 0 and codes 0; one that holds an infinity or a NaN
 * has scale NaN and codes 0.  codes [M][ldq], any ldq >= K; columns K .. ldq - 1 are left as they
 * are. */
gemm_status_t gemm_run_quantize_int8(const void *X, void *codes, float *scale, int64_t M,
                                     int64_t K, int64_t ldx, int64_t ldq, int in_dtype,
                                     hipStream_t stream);

/* C = act(alpha y + beta C_old + bias), y[m][n] = scale_a[m] scale_b[n] sum_k A[m][k]
 * B[n][k], A [M][K] and B [N][K] INT8 (-128 .. 127), C [M][N] of out_dtype; epi as gemm_run_ex's
 * (NULL: the identity).  The sum is exact (INT32, K splits and all), taken to FP32, multiplied
 * by scale_a[m] and then by scale_b[n].
 *   scales_a  M, or 1: one scale for all rows;  scales_b  N, or 1
 *   K % 16 == 0, K < 2^17 */
gemm_status_t gemm_int8_workspace(int64_t M, int64_t N, int64_t K, int64_t *bytes);
gemm_status_t gemm_run_int8(const void *A, const void *B, void *C, int64_t M, int64_t N, int64_t K,
                            int64_t lda, int64_t ldb, int64_t ldc, int out_dtype,
                            const float *scale_a, int64_t scales_a, const float *scale_b,
                            int64_t scales_b, const gemm_epilogue_t *epi, void *workspace,
                            int64_t workspace_bytes, hipStream_t stream);

/* The orthogonalized update of a stack of weights: for each matrix G [m][n] (GEMM_BF16,
 * GEMM_FP16 or GEMM_FP32; rows of ldg elements, matrices g_step apart), X = G / (||G|| + eps)
 * with the Frobenius norm, then for each step i
 *   X = a X + b (X X^T) X + c (X X^T)^2 X,   (a, b, c) = coefficients[3 i .. 3 i + 2]
 * (for m > n with X^T X on the other side, which is the same), so that every singular
 * value s of X becomes a s + b s^3 + c s^5.  U [m][n] of out_dtype, rows of ldu, matrices u_step
 * apart; its matrices must not overlap (it may be G).  `coefficients` is a host array, read in the call.
 *
 * The norm is an FP64 sum; X is kept as the sum of two FP16 values (22 bits, scaled); the
 * products run on the first of them with FP32 sums.  With coefficients that keep the singular values below 2, U is about
 * 1e-3 of the exact iteration off (relative, of the whole matrix; 4e-3 where half of the
 * singular values are zero), so that an FP32 U is no more exact than that.  An infinity or NaN in G makes its
 * matrix NaN.  steps = 0: X.  batch <= 65535, m and n at most 2^20; any ldg >= n, ldu >= n. */
gemm_status_t gemm_orthogonalize_workspace(int64_t batch, int64_t m, int64_t n, int64_t *bytes);
gemm_status_t gemm_run_orthogonalize(const void *G, void *U, int64_t batch, int64_t m, int64_t n,
                                     int64_t ldg, int64_t ldu, int64_t g_step, int64_t u_step,
                                     int in_dtype, int out_dtype, int64_t steps,
                                     const float *coefficients, double eps, void *workspace,
                                     int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_LAYER_H */
