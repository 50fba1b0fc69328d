/*
 * rlk/step_ops.h — C ABI of the operators that stand before and behind the
 * LM head of rlk.h in a training step:
 *
 *   layer_norm, rms_norm   the norm that makes the hidden states h;
 *   embed                  token embeddings with a scale, and the gradient
 *                          of their table: dense, or added to one that is
 *                          there (the LM head's grad_W of a tied weight);
 *   grad_norm, clip_grads  the norm of a list of gradients, and their
 *                          scaling to a largest norm.
 *
 * The conventions of rlk.h hold (device pointers, owned by the caller; work
 * is only enqueued on `stream`, nothing is allocated or synchronised; status
 * codes), except:
 *   - arrays need the alignment of their elements only, ws 16 bytes;
 *   - H is any width in [1, 65536];
 *   - T <= 2^23; with T == 0 only gradients that are sums over the rows are
 *     written (zeros).
 * The current device must be the one the arrays live on.  Types are
 * RLK_DT_F32 and RLK_DT_BF16.
 *
 * Everything is computed in fp32 (the gradients' norm in fp64) and rounded
 * once to the output's type.  Sums have a fixed order: repeated runs are
 * bit-identical.  A row's y, mean, rstd, out and grad_x depend only on that
 * row, whatever the batch, its strides or alignment; an embedding's gradient
 * row depends only on the rows of g that have its token, in their order.
 */
#ifndef RLK_STEP_OPS_H_
#define RLK_STEP_OPS_H_

#include "../rlk.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { RLK_SOP_NORM_BWD = 0, RLK_SOP_EMBED_BWD = 1, RLK_SOP_GRADS = 2 };

/* Workspace bytes of rlk_*_norm_bwd (T, H), of rlk_embed_bwd (T, H, V), and of
 * rlk_grad_norm and rlk_clip_grads for T tensors (H and V are not read).  0 for
 * invalid arguments. */
size_t rlk_step_workspace_bytes(int32_t op, int64_t T, int64_t H, int64_t V);

/* Layer norm over rows of H elements:
 *   mean = sum(x) / H,  rstd = 1 / sqrt(sum((x - mean)^2) / H + eps),
 *   y = (x - mean) rstd weight + bias
 *   x       [T,H] of x_dtype, row t at x + t * ldx elements (ldx >= 0; 0: every
 *           row is the same one)
 *   weight, bias  [H] of w_dtype; either may be NULL (ones, zeros)
 *   y       [T,H] out of y_dtype
 *   mean, rstd  fp32 [T] out, what the backward needs; either may be NULL
 * eps >= 0 and finite.  The sums are fp32.  The sum of x may pass 3.4e38; a row
 * whose squares about the mean add up past it has rstd 0, so its y is bias, or 0
 * (NaN where x - mean itself passes it).  A NaN or infinite element reaches its
 * own row only. */
rlk_status rlk_layer_norm_fwd(const void* x, int32_t x_dtype, int64_t ldx, const void* weight, const void* bias,
                              int32_t w_dtype, int64_t T, int64_t H, float eps, void* y, int32_t y_dtype, float* mean,
                              float* rstd, void* stream);

/* Gradient of sum(g * y), with n = (x - mean) rstd and gw = g weight:
 *   grad_x = rstd (gw - sum(gw) / H - n sum(gw n) / H)
 *   grad_weight = sum_t g n,  grad_bias = sum_t g
 *   g       [T,H] of g_dtype, row stride ldg >= 0
 *   grad_x  [T,H] out of x_dtype; may be NULL
 *   grad_weight, grad_bias  [H] out of grad_dtype; either may be NULL */
rlk_status rlk_layer_norm_bwd(const void* x, int32_t x_dtype, int64_t ldx, const void* weight, int32_t w_dtype,
                              const float* mean, const float* rstd, const void* g, int32_t g_dtype, int64_t ldg,
                              int64_t T, int64_t H, void* grad_x, void* grad_weight, void* grad_bias,
                              int32_t grad_dtype, void* ws, size_t ws_bytes, void* stream);

/* RMS norm: rstd = 1 / sqrt(sum(x^2) / H + eps), y = x rstd weight; rstd and y are
 * 0 where the squares add up past 3.4e38. */
rlk_status rlk_rms_norm_fwd(const void* x, int32_t x_dtype, int64_t ldx, const void* weight, int32_t w_dtype,
                            int64_t T, int64_t H, float eps, void* y, int32_t y_dtype, float* rstd, void* stream);

/* n = x rstd, gw = g weight: grad_x = rstd (gw - n sum(gw n) / H),
 * grad_weight = sum_t g n. */
rlk_status rlk_rms_norm_bwd(const void* x, int32_t x_dtype, int64_t ldx, const void* weight, int32_t w_dtype,
                            const float* rstd, const void* g, int32_t g_dtype, int64_t ldg, int64_t T, int64_t H,
                            void* grad_x, void* grad_weight, int32_t grad_dtype, void* ws, size_t ws_bytes,
                            void* stream);

/* out[t] = scale E[ids[t]].
 *   ids  [T] token ids, int32 (id_bytes 4) or int64 (8); rows equal to
 *        ignore_index are zero
 *   E    [V,H] of E_dtype;  out  [T,H] of out_dtype
 * A row whose id lies outside [0, V) is NaN.  scale is finite. */
rlk_status rlk_embed_fwd(const void* ids, int32_t id_bytes, const void* E, int32_t E_dtype, int64_t T, int64_t H,
                         int64_t V, int64_t ignore_index, float scale, void* out, int32_t out_dtype, void* stream);

/* grad_E[v] = scale * sum over t with ids[t] == v of g[t]: rows ascending in runs
 * of 16 from the token's first row on, then these sums, in an order that goes by
 * their number alone.
 *   g       [T,H] of g_dtype, row stride ldg >= 0
 *   grad_E  [V,H] of grad_dtype.  accumulate == 0: written whole, zero rows for
 *           tokens that do not occur.  accumulate == 1: the sum is added (in
 *           fp32) to the rows that occur, the others are left as they are.
 * Rows of ignore_index, and rows whose id lies outside [0, V), reach no row of
 * grad_E. */
rlk_status rlk_embed_bwd(const void* ids, int32_t id_bytes, const void* g, int32_t g_dtype, int64_t ldg, int64_t T,
                         int64_t H, int64_t V, int64_t ignore_index, float scale, void* grad_E, int32_t grad_dtype,
                         int32_t accumulate, void* ws, size_t ws_bytes, void* stream);

/* norm = sqrt of the sum of squares over all elements of n tensors, taken in
 * fp64 and rounded once.
 *   grads, sizes, dtypes  HOST arrays of n: device pointers, element counts
 *          (0 .. 2^36) and types; read before the call returns
 *   norm   fp32 [1] out
 * 0 <= n <= 2^20. */
rlk_status rlk_grad_norm(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int32_t n, float* norm,
                         void* ws, size_t ws_bytes, void* stream);

/* The norm as above, and out = c grads with c = max_norm / norm (fp64, rounded
 * to fp32) where norm > max_norm, else 1; each product rounded once to the
 * output's type.  The norm's fp64 value is what counts: one that only fp32
 * cannot hold is stored as infinity, and scales as any other.  A NaN norm makes c
 * NaN; an infinite gradient, c = 0 (and NaN where a gradient is infinite).
 *   out, out_dtypes  HOST arrays of n; out[i] may be grads[i] with its type.
 * Arrays that overlap otherwise are refused (RLK_ERR_BAD_ARG): an output with
 * another output, or with a gradient that is not its own.
 * max_norm >= 0 (+inf: nothing is scaled). */
rlk_status rlk_clip_grads(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int32_t n,
                          float max_norm, void* const* out, const int32_t* out_dtypes, float* norm, void* ws,
                          size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RLK_STEP_OPS_H_ */
