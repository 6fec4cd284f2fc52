/*
 * gemm_rows.h -- C ABI of the MI355X (gfx950) products whose weight depends on
 * the row: a shared projection with low-rank adapters picked per row, the
 * router that picks experts per row, and the experts' products over its rows.
 * Built as libgemm_rows.so, beside gemm_nt.h's library, whose types, status
 * codes and epilogue it uses.
 *
 * What picks the weight (adapter ids, expert offsets) is read on the device by
 * the kernels: no call copies it to the host, so every call can be captured
 * into a HIP graph and replayed with other ids in the same buffers.  An id or
 * offset that is out of range never leads outside a buffer; each entry point
 * says what it means.
 *
 * Storage, types, rounding: row-major with element strides, BF16 or FP16
 * operands (all of one call's 16-bit operands share the type), FP32 sums,
 * results rounded once to nearest even.  Limits as gemm_run's: sizes below
 * 2^31 (rows of gemm_run_lora and its backward below 2^30), fewer than 2^23
 * output tiles, leading dimensions of operands below 2^22 and multiples of 8,
 * operand bases 16-byte aligned.  For given arguments every call on the same device
 * returns the same bits.
 *
 * Workspaces: no handle; a call that needs one takes a device workspace of the
 * caller's, 256-byte aligned and at least as large as the matching *_workspace function
 * says for the same sizes.  Nothing needs to be in it before a call, and
 * nothing is kept in it between calls.  Two calls that may run concurrently
 * (different streams, two graphs' replays) need workspaces of their own.  A
 * call allocates nothing and only enqueues work on `stream`, for the device
 * that is current.
 *
 * Errors: GEMM_ERR_INVALID_ARG for null pointers, negative sizes, leading
 * dimensions that are too small, unknown modes and a workspace that is too
 * small; GEMM_ERR_UNSUPPORTED for types and sizes outside the limits;
 * GEMM_ERR_MISALIGNED; GEMM_ERR_HIP.  On an error nothing is enqueued, but for
 * GEMM_ERR_HIP, after which part of a call's launches may be.
 */
#ifndef GEMM_ROWS_H
#define GEMM_ROWS_H

#include <stdint.h>

#include "gemm_nt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Low-rank adapters: adapter a is the pair of A_a (rank rows of a_ld elements,
 * at A + a * a_stride) and B_a (N rows of b_ld elements, at B + a * b_stride)
 * with the FP32 factor scale[a].  ids[m] is row m's adapter; a value outside
 * [0, num_adapters) (customarily -1) means none.  rank must be a multiple of 8
 * up to 128; adapters of smaller rank are padded with zero rows of A (and any
 * finite columns of B).  num_adapters = 0 or rank = 0: no row has an adapter.
 *   a_ld >= K, b_ld >= rank, both and the strides multiples of 8;
 *   rank * a_ld and N * b_ld below 2^30 */
typedef struct {
    const void *A;
    const void *B;
    const float *scale;     /* device, num_adapters values */
    const int32_t *ids;     /* device, M values */
    int64_t num_adapters, rank;
    int64_t a_stride, a_ld;
    int64_t b_stride, b_ld;
} gemm_adapters_t;

/* Y[m,:] = act(alpha (X[m,:] W^T + s_a (X[m,:] A_a^T) B_a^T) + beta Y_old + bias),
 * a = ids[m]: X [M][K], W [N][K], Y [M][N] of out_dtype (GEMM_BF16, GEMM_FP16,
 * GEMM_FP32); epi as gemm_run_ex's (NULL: the identity).  The adapters' part is
 * added to the projection's FP32 sums, so Y is rounded once.  The low-rank
 * values X A_a^T are FP32 sums; scaled, they enter the second product as the
 * sum of two values of the operands' type (three where BF16 operands have an FP32
 * result), of FP16 operands in units of a power of two of each row's, so that small and
 * large ones keep their bits: to 2^-22 of the largest of their 16 ranks (2^-40 of the row's
 * largest, and 2^-85), and up to 2^75 (above it the result is infinite or NaN).
 *   K % 8 == 0 (else GEMM_ERR_UNSUPPORTED).  K = 0: the epilogue of zero. */
gemm_status_t gemm_lora_workspace(int64_t M, int64_t N, int64_t K, int64_t num_adapters,
                                  int64_t rank, int64_t *bytes);
gemm_status_t gemm_run_lora(const void *X, const void *W, void *Y, int64_t M, int64_t N, int64_t K,
                            int64_t ldx, int64_t ldw, int64_t ldy, int in_dtype, int out_dtype,
                            const gemm_adapters_t *adapters, const gemm_epilogue_t *epi,
                            void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* Gradients of Y = X W^T + s_a (X A_a^T) B_a^T for dY [M][N], W being frozen:
 *   dX[m,:] = dY[m,:] W + s_a (dY[m,:] B_a) A_a          [M][K], dx_dtype
 *   dA_a    = s_a sum_{m: ids[m] = a} (dY[m,:] B_a)^T X[m,:]   [adapter][rank][K]
 *   dB_a    = s_a sum_{m: ids[m] = a} dY[m,:]^T (X[m,:] A_a^T) [adapter][N][rank]
 * dY B_a and X A_a^T are FP32 sums.  They enter dX as above; dA and dB take
 * them, scaled, to 24 bits in FP32's range, whatever their size.
 * dA and dB are contiguous, of grad_dtype, and written whole: adapters without
 * a row get zeros.  dX may be NULL (not computed), and so may dA and dB, both
 * or neither.  K % 8 == 0, N % 8 == 0 and num_adapters <= 1024 (else
 * GEMM_ERR_UNSUPPORTED).  M = 0 writes zeros to dA and dB. */
gemm_status_t gemm_lora_backward_workspace(int64_t M, int64_t N, int64_t K, int64_t num_adapters,
                                           int64_t rank, int64_t *bytes);
gemm_status_t gemm_run_lora_backward(const void *dY, const void *X, const void *W, void *dX,
                                     void *dA, void *dB, int64_t M, int64_t N, int64_t K,
                                     int64_t lddy, int64_t ldx, int64_t ldw, int64_t lddx,
                                     int in_dtype, int dx_dtype, int grad_dtype,
                                     const gemm_adapters_t *adapters, void *workspace,
                                     int64_t workspace_bytes, hipStream_t stream);

/* What a router call writes; every pointer is required (k = top_k).
 *   ids      [T][k]    the chosen experts, by falling logit, or -1
 *   weights  [T][k]    their weights, FP32 (0 where ids is -1)
 *   counts   [E]       how many (token, choice) pairs chose each expert
 *   offsets  [E + 1]   exclusive prefix sums of counts
 *   order    [T k]     the pairs t k + j sorted by expert, in order within
 *                      one; those with ids = -1 come last, behind offsets[E]
 *   tokens   [1]       n, the tokens that were routed (below)
 *   loss     [1]       the balance loss, FP32 */
typedef struct {
    int32_t *ids;
    float *weights;
    int32_t *counts;
    int32_t *offsets;
    int32_t *order;
    int32_t *tokens;
    float *loss;
} gemm_routing_t;

/* Top-k router over logits [T][E] (rows of ld elements; BF16, FP16 or FP32).
 * p = softmax over a token's logits; its top_k largest logits are its choices,
 * equal ones by the lower expert index (-0 and +0 are equal).  A logit of -inf
 * closes an expert to the token: it is never chosen, and a token with fewer than
 * top_k open experts has -1 in the places left.  mask (one byte per token, 0:
 * padding; NULL: none) takes tokens out; they, and tokens without an open
 * expert, are not routed: ids -1, weights 0, p = 0.
 * (p is FP32: below 2^-126 it may be zero.)
 *   weights = p of the choice, divided by the choices' sum where renormalize
 *   loss    = E sum_e f_e P_e, f_e = counts[e] / (n top_k),
 *             P_e = (sum over routed tokens of p_e) / n; 0 for n = 0
 * (1 for an even routing).  A +inf or NaN logit makes its token's p NaN, and so
 * the loss; the token's choices are then still distinct experts (NaN ranks
 * as the lowest finite logit).  1 <= top_k <= min(E, 64), E <= 1024,
 * T top_k < 2^31 (else GEMM_ERR_UNSUPPORTED); any ld >= E. */
gemm_status_t gemm_route_workspace(int64_t T, int64_t E, int64_t top_k, int64_t *bytes);
gemm_status_t gemm_run_route(const void *logits, const uint8_t *mask, int64_t T, int64_t E,
                             int64_t ld, int64_t top_k, int renormalize, int dtype,
                             const gemm_routing_t *out, void *workspace, int64_t workspace_bytes,
                             hipStream_t stream);

/* Gradient of gemm_run_route's weights and loss in the logits: dlogits [T][E]
 * (rows of ldd elements, the logits' type) from grad_weights [T][top_k] FP32
 * and grad_loss [1] FP32 (either may be NULL: zero).  `in` is that call's
 * output (its order and offsets are not read); counts enter the loss as
 * constants.  Tokens that were not routed get zeros, as do closed experts. */
gemm_status_t gemm_run_route_backward(const void *logits, const gemm_routing_t *in,
                                      const float *grad_weights, const float *grad_loss,
                                      void *dlogits, int64_t T, int64_t E, int64_t ld, int64_t ldd,
                                      int64_t top_k, int renormalize, int dtype,
                                      hipStream_t stream);

/* Rows of no expert, before the first expert's and behind the last's: left as they
 * are, or set to zero. */
typedef enum { GEMM_TAIL_KEEP = 0, GEMM_TAIL_ZERO = 1 } gemm_tail_t;

/* The experts' products over rows sorted by expert: for offsets[e] <= i <
 * offsets[e + 1], C[i,:] = X[i,:] op(W_e), X [rows][K], C [rows][N], W_e at
 * W + e * w_stride.  layout_w GEMM_K_MAJOR: W_e is [N][ldw], op(W_e) = W_e^T
 * (the forward product); GEMM_MN_MAJOR: W_e is [K][ldw], op(W_e) = W_e (with
 * X the output gradient, the input gradient of the former).
 *   offsets  device, num_experts + 1 values; read as clamped to [0, rows] and
 *            to their running maximum, so a decreasing or too large one leaves
 *            its expert without rows
 *   tail     gemm_tail_t, for the rows before offsets[0] and behind the last
 *            expert's
 *   num_experts <= 1024; K % 8 == 0; rows = 0 or N = 0 enqueues nothing */
gemm_status_t gemm_run_routed(const void *X, const void *W, void *C, const int32_t *offsets,
                              int64_t rows, int64_t N, int64_t K, int64_t num_experts, int64_t ldx,
                              int64_t ldw, int64_t w_stride, int64_t ldc, int layout_w,
                              int in_dtype, int out_dtype, int tail, hipStream_t stream);

/* Weight gradients of the experts: dW_e = sum over e's rows i of dY[i,:]^T X[i,:],
 * dY [rows][N], X [rows][K], dW [num_experts][N][K] contiguous, of out_dtype,
 * written whole (zeros for an expert without rows).  Offsets as above.
 * N % 8 == 0 and K % 8 == 0. */
gemm_status_t gemm_run_routed_wgrad(const void *dY, const void *X, void *dW,
                                    const int32_t *offsets, int64_t rows, int64_t N, int64_t K,
                                    int64_t num_experts, int64_t lddy, int64_t ldx, int in_dtype,
                                    int out_dtype, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_ROWS_H */
