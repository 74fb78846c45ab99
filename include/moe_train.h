/*
 * moe_train.h — C ABI of the operators that training an MoE block adds to the
 * forward of moe.h, in the same library (libmoe_gb300.so):
 *
 *   moe_layer_norm              layer norm of the token rows in front of the router
 *   moe_layer_norm_backward     ... its gradient, with the reduction of the weights' gradients
 *   moe_balance_loss            load-balance loss of the router and per-expert counts
 *   moe_balance_loss_backward   ... its gradient with respect to the router's output
 *   moe_checkpoint_pack         bf16 rows to an 8-bit checkpoint
 *   moe_checkpoint_unpack       ... and back
 *   moe_silu_mul_checkpoint     z = silu(y0) * y1, keeping y0 and y1 as an 8-bit checkpoint
 *   moe_silu_mul_backward       the gradient of silu_mul, read from that checkpoint
 *   moe_grouped_weight_grad     the experts' weight gradients dW[e] = dY_e^T X_e
 *
 * The conventions of moe.h hold: device pointers owned by the caller, no
 * allocation, everything asynchronous on `stream`, status codes for argument
 * errors, MOE_DEVERR_* bits for what only the GPU can see, identical bytes for
 * identical inputs on the same device.  The sizes that need not be multiples of
 * 16 are named below.  Outputs must not overlap inputs.
 */
#ifndef MOE_GB300_TRAIN_H
#define MOE_GB300_TRAIN_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* -------------------------------------------------------------- layer norm */

/*
 * For every token t < Tv:
 *   mean[t] = (1/D) sum_d x[t, d]
 *   rstd[t] = 1 / sqrt((1/D) sum_d (x[t, d] - mean[t])^2 + eps)
 *   y[t, d] = (x[t, d] - mean[t]) * rstd[t] * gamma[d] + beta[d]
 * in fp32 (the variance from the centred values), y rounded once.
 *
 * x [T, D] of dtype MOE_DTYPE_BF16 or MOE_DTYPE_F32, row stride ldx >= D
 * elements; y [T, D] of the same dtype, contiguous; gamma [D] and beta [D]
 * (nullable: 0) of weight_dtype, one of the same two.
 * mean, rstd fp32 [T], each nullable: what the backward pass takes.
 * num_valid_tokens: device int32 Tv (NULL: T); a value outside [0, T] is
 * clamped and flagged.  Rows t >= Tv of the outputs are not written.
 * Any 1 <= D <= 16384 (larger: MOE_ERR_UNSUPPORTED), any element alignment;
 * eps >= 0 and finite.  T == 0 or D == 0 is a no-op.
 */
int moe_layer_norm(const void* x, int64_t ldx, int T, int D, int dtype, const void* gamma, const void* beta,
                   int weight_dtype, float eps, const int32_t* num_valid_tokens, void* y, float* mean,
                   float* rstd, cudaStream_t stream);

/*
 * The gradient: with xh = (x - mean) * rstd and g = dy * gamma, for t < Tv
 *   dx[t, d] = rstd[t] * (g - (1/D) sum_d g - xh * (1/D) sum_d g xh) [+ residual_grad[t, d]]
 *   dgamma[d] = sum_t dy[t, d] * xh[t, d],   dbeta[d] = sum_t dy[t, d]
 * in fp32.  x, ldx, dtype, gamma, weight_dtype, num_valid_tokens: as in
 * moe_layer_norm; mean, rstd: its outputs.  dy, dx, residual_grad (nullable: the
 * gradient that reaches x past the norm, added before the one rounding) [T, D]
 * of dtype, contiguous.  dgamma, dbeta (nullable) fp32 [D], overwritten; both
 * are zero when Tv == 0 (T == 0 included).
 * ws: device workspace of moe_layer_norm_backward_workspace_size bytes, 16-byte
 * aligned; its contents on entry do not matter.
 */
int moe_layer_norm_backward_workspace_size(int T, int D, size_t* bytes);
int moe_layer_norm_backward(const void* dy, const void* x, int64_t ldx, int T, int D, int dtype, const void* gamma,
                            int weight_dtype, const float* mean, const float* rstd, const int32_t* num_valid_tokens,
                            const void* residual_grad, void* dx, float* dgamma, float* dbeta, void* ws,
                            size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------ balance loss */

/* What the router's output a[t, e] is, and how it becomes a distribution p over experts. */
#define MOE_BALANCE_SCORES 0  /* scores >= 0 (moe_router_scores): p = a / sum_e a, 0 where the sum is 0 */
#define MOE_BALANCE_SOFTMAX 1 /* logits: p = softmax(a); a row of -inf alone has p = 0 */
/* logits: s = sigmoid(a), p = s / sum_e s.  The sum may be far below fp32's least number; a row
 * whose logits are all below -700 (masked by the type's lowest value or -inf) has p = 0. */
#define MOE_BALANCE_SIGMOID 2

/*
 * The load-balance loss of a top-k router over the valid tokens t < Tv:
 *   counts[e]     = number of tokens whose top_k largest a[t, .] include e
 *   mean_probs[e] = (1/Tv) sum_t p[t, e]
 *   loss[0]       = coefficient * sum_e f_e * mean_probs[e],  f_e = E * counts[e] / (top_k * Tv)
 * which is `coefficient` for a balanced router.  Tv == 0: counts, mean_probs
 * and loss are 0.
 *
 * scores      [T, E], element (t, e) at scores + t * stride_t + e * stride_e,
 *             MOE_DTYPE_BF16 or MOE_DTYPE_F32.  NaN is undefined, as in moe_route.
 * counts_in   device int32 [>= E], nullable: the counts of moe_route or
 *             moe_router_route for the same tokens and top_k.  Given, nothing is
 *             selected here and counts_out is not used.
 * counts_out  device int32 [E + 1], required when counts_in is NULL: the
 *             selection is moe_route's (equal values to the lower expert), made on
 *             the values of `scores`; counts_out[E] = Tv * top_k.
 * mean_probs  fp32 [E]; loss fp32 [1].
 * 1 <= top_k <= E <= 1024.
 * ws: device workspace of moe_balance_loss_workspace_size bytes, 16-byte
 * aligned; its contents on entry do not matter.  One workspace serves one call
 * at a time.
 */
int moe_balance_loss_workspace_size(int T, int E, size_t* bytes);
int moe_balance_loss(const void* scores, int scores_dtype, int64_t stride_t, int64_t stride_e, int T, int E,
                     int top_k, int kind, float coefficient, const int32_t* num_valid_tokens,
                     const int32_t* counts_in, int32_t* counts_out, float* mean_probs, float* loss, void* ws,
                     size_t ws_bytes, cudaStream_t stream);

/*
 * Its gradient with respect to scores, the counts being constants: with
 * q_t = sum_e f_e p[t, e] and w = dloss * coefficient / Tv, for t < Tv
 *   SCORES:  dscores[t, e] = w (f_e - q_t) / sum_e a          (0 where the sum is 0)
 *   SOFTMAX: dscores[t, e] = w (f_e - q_t) p[t, e]
 *   SIGMOID: dscores[t, e] = w (f_e - q_t) p[t, e] (1 - s[t, e])
 * counts: device int32 [>= E] (moe_balance_loss's counts, or moe_route's).
 * dloss: device fp32 scalar, nullable: 1.  dscores [T, E] contiguous, of
 * scores_dtype; overwritten, or with accumulate != 0 added to (in fp32, one
 * rounding).  Rows t >= Tv are not written.
 */
int moe_balance_loss_backward(const void* scores, int scores_dtype, int64_t stride_t, int64_t stride_e, int T, int E,
                              int top_k, int kind, float coefficient, const int32_t* num_valid_tokens,
                              const int32_t* counts, const float* dloss, void* dscores, int accumulate,
                              cudaStream_t stream);

/* ------------------------------------------------------ 8-bit checkpoints */

/*
 * An 8-bit checkpoint of bf16 rows v [a, W]: codes [a, W] e4m3 and one exponent
 * byte per block of MOE_CHECKPOINT_BLOCK columns of a row, exponents
 * [a, ceil(W / 128)] (the last block of a row may be short).  For a block with
 * m = max |v| over its finite values,
 *   e    = the least integer with m <= 448 * 2^e, within [-100, 119] (-100 for m = 0)
 *   code = e4m3(v * 2^-e), round to nearest even, saturating; NaN for NaN and +-inf
 *   byte = e + 127
 * and the value kept is code * 2^e, which bf16 holds exactly: what reads a
 * checkpoint as bf16 loses nothing more.
 *
 * x bf16 [a, W] with row stride ld elements; W % 16 == 0, ld % 8 == 0, 16-byte
 * aligned bases (MOE_ERR_UNSUPPORTED).  valid_rows: device int32 row count
 * (NULL: a; clamped to [0, a] and flagged); rows at or past it are not written.
 */
#define MOE_CHECKPOINT_BLOCK 128
int moe_checkpoint_pack(const void* x, int64_t ld, int a, int W, const int32_t* valid_rows, void* codes,
                        uint8_t* exponents, cudaStream_t stream);
int moe_checkpoint_unpack(const void* codes, const uint8_t* exponents, int a, int W, const int32_t* valid_rows,
                          void* x, cudaStream_t stream);

/*
 * moe_silu_mul (bit for bit: z [a, H] bf16 from x0, x1 with row stride ld)
 * that also keeps its input as a checkpoint of two halves: codes [a, 2H] (x0's
 * H columns, then x1's), exponents [a, 2 * ceil(H / 128)] (x0's blocks, then
 * x1's; blocks do not cross from one half to the other).
 */
int moe_silu_mul_checkpoint(const void* x0, const void* x1, int64_t ld, int a, int H, const int32_t* valid_rows,
                            void* z, void* codes, uint8_t* exponents, cudaStream_t stream);

/*
 * The gradient of z = silu(y0) * y1 at the kept values y0, y1 of such a
 * checkpoint; with s = sigmoid(y0), in fp32:
 *   dy[r, j]     = bf16(dz y1 s (1 + y0 (1 - s)))
 *   dy[r, H + j] = bf16(dz y0 s)
 *   z[r, j]      = bf16(y0 s y1)        (z nullable: what the gradient of w2 takes)
 * dz [a, H] bf16, dy [a, 2H] bf16, z [a, H] bf16, contiguous.
 */
int moe_silu_mul_backward(const void* codes, const uint8_t* exponents, const void* dz, int a, int H,
                          const int32_t* valid_rows, void* dy, void* z, cudaStream_t stream);

/* ---------------------------------------------------------- weight gradient */

/*
 * The weight gradients of a grouped GEMM y_r = w[e] x_r (moe_grouped_gemm):
 *   dw[e, n, k] = sum over the rows r of expert e of dy[r, n] * x[r, k]   (fp32 accumulation)
 * with expert e's rows as in moe_grouped_gemm: [off_e, off_e + counts[e]).  An
 * expert without rows gets zeros (nothing is added with accumulate).
 *
 * dy [a_max, N] bf16.  x [a_max, K] bf16 with x_exponents NULL, or the e4m3
 * codes of a checkpoint with its exponents [a_max, ceil(K / 128)].
 * dw [E, N, K] of dw_dtype: MOE_DTYPE_BF16 (one rounding), or MOE_DTYPE_F32,
 * which accumulate != 0 adds to (a gradient over several micro-batches);
 * accumulate with bf16 is MOE_ERR_INVALID.
 * counts [E] device int32: negative entries count as 0 and a sum past a_max is
 * cut there; both are flagged (MOE_DEVERR_BAD_COUNT).  Rows past the sum are not
 * read into any result, whatever they hold.
 * N and K multiples of 16, E <= 1024 (MOE_ERR_UNSUPPORTED).
 * ws: device workspace of moe_grouped_weight_grad_workspace_size bytes (x_dtype
 * MOE_DTYPE_BF16 or MOE_DTYPE_E4M3; it may be 0: ws may then be NULL), 256-byte
 * aligned; its contents on entry do not matter.  It holds the unpacked rows of a
 * checkpoint, and fp32 parts of dw where few tiles make it worth cutting long
 * experts' rows; the parts are added in order.
 */
int moe_grouped_weight_grad_workspace_size(int E, int a_max, int N, int K, int x_dtype, size_t* bytes);
int moe_grouped_weight_grad(const void* dy, const void* x, const uint8_t* x_exponents, const int32_t* counts, int E,
                            int a_max, int N, int K, void* dw, int dw_dtype, int accumulate, void* ws,
                            size_t ws_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_TRAIN_H */
