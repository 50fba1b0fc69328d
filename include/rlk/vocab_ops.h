/*
 * rlk/vocab_ops.h — C ABI of the operators on the whole next-token
 * distribution of an LM head, beside the selected log-probability of rlk.h:
 *
 *   linear_logp_top   the selected log-probability with the entropy of the
 *                     distribution and its K most likely tokens, and the
 *                     gradient of log-probability and entropy;
 *   linear_distill    the divergence KL(q || p) from a teacher's distribution
 *                     q over its kept tokens, and its gradient.
 *
 * Both go from the bf16 hidden states h [T,H] and the bf16 weight W [V,H] to
 * their result without a [T,V] logits tensor of the caller's, on the tile
 * engine of rlk.h and under its numerical contract: logits are the same MFMA
 * chains, statistics are folded in the same fixed order, and a row's results
 * depend only on that row.  Repeated runs are bit-identical; a row's results
 * (grad_h included) do not change with the batch it is in.
 *
 * The conventions of rlk.h hold (device pointers to contiguous arrays, owned
 * by the caller; work is only enqueued on `stream`, nothing is allocated or
 * synchronised; outputs are overwritten; H % 64 == 0; status codes), except:
 *   - h, W, ws, grad_h and grad_W are 16-byte aligned; arrays of rows or of
 *     rows and slots need the alignment of their elements (4 bytes);
 *   - T <= 2^23; T == 0 launches nothing but the zeroing of a wanted grad_W.
 * The current device must be the one the arrays live on.
 */
#ifndef RLK_VOCAB_OPS_H_
#define RLK_VOCAB_OPS_H_

#include "../rlk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The largest K (alternatives, or teacher's tokens, of a row). */
#define RLK_MAX_K 128

enum { RLK_VOP_TOP_FWD = 0, RLK_VOP_TOP_BWD = 1, RLK_VOP_DISTILL_FWD = 2, RLK_VOP_DISTILL_BWD = 3 };

/* Workspace bytes of an operator (RLK_VOP_*).  0 for invalid arguments.
 * RLK_VOP_TOP_BWD does not depend on K (pass any valid one).
 *
 * The vocabulary is processed in groups of splits: the forward of
 * linear_logp_top keeps a group's fp32 logits (K > 0), the backwards a
 * group's bf16 dz, each within the budget of rlk_workspace_bytes
 * (RLK_DZ_BUDGET_MB; no result bit depends on it).  Up to 128 rows both
 * forwards keep all logits where the budget holds them.  The backwards also
 * hold grad_h in fp32 parts, 4 T H floats of them or more for narrow heads
 * (8 at H = 2048, 32 at 512, V = 151936). */
size_t rlk_vocab_workspace_bytes(int32_t op, int64_t T, int64_t H, int64_t V, int64_t K);

/* Selected log-probability, entropy and top alternatives, z = h W^T:
 *   logp[t]    = z[t, y_t] - lse[t]               (the bits of rlk_linear_logp_fwd)
 *   entropy[t] = -sum_v p_v log p_v               p = softmax(z[t])
 *   top_ids[t, k], top_logp[t, k], k < K: the K largest logits of the row,
 *                best first, ties to the lowest id, and their log p
 *   y         int32 [T]   target ids; rows equal to ignore_index are inactive:
 *                         logp = lse = entropy = 0, ids -1, top_logp -inf
 *   lse       fp32 [T] out, may be NULL
 *   top_logp  fp32 [T,K] out, top_ids int32 [T,K] out; slots past V hold -1
 *                         and -inf; may be NULL when K == 0
 * 0 <= K <= RLK_MAX_K.  A target outside [0, V) gives NaN in the row's logp;
 * its entropy and alternatives are those of the row.  A logit of -inf has
 * probability 0 and is an alternative only after all others (grad_h has the
 * NaN of 0 times an infinite weight; a finite mask keeps it defined).  A NaN
 * or +inf logit makes logp, lse, entropy and top_logp NaN; NaN is never an
 * alternative, and a row of nothing but NaN has none (-1 and -inf). */
rlk_status rlk_linear_logp_top_fwd(const void* h, const void* W, const int32_t* y, int64_t T, int64_t H, int64_t V,
                                   int32_t ignore_index, int64_t K, float* logp, float* lse, float* entropy,
                                   float* top_logp, int32_t* top_ids, void* ws, size_t ws_bytes, void* stream);

/* Gradient of sum_t g[t] logp[t] + g_entropy[t] entropy[t]:
 *   dz_v = g [v = y] - p_v (g + g_entropy (entropy + z_v - lse)),
 *   grad_h = dz W, grad_W = dz^T h.
 *   lse, entropy   fp32 [T]  the forward's
 *   g, g_entropy   fp32 [T]  upstream gradients; either may be NULL (zero)
 *   grad_h  bf16 [T,H] out, may be NULL; zero rows for inactive rows
 *   grad_W  [V,H] out of grad_W_dtype (RLK_DT_F32, or RLK_DT_BF16: each fp32
 *           sum rounded once), may be NULL
 * dz is rounded to bf16 once, as in rlk_linear_logp_bwd (up to 2^-8 of each
 * dz; where one dz dominates, with one or two active rows, that scales whole
 * rows of the gradients); sums are fp32.  An active row whose target lies
 * outside [0, V) makes its grad_h row and grad_W NaN. */
rlk_status rlk_linear_logp_top_bwd(const void* h, const void* W, const int32_t* y, const float* lse,
                                   const float* entropy, const float* g, const float* g_entropy, int64_t T, int64_t H,
                                   int64_t V, int32_t ignore_index, void* grad_h, void* grad_W, int32_t grad_W_dtype,
                                   void* ws, size_t ws_bytes, void* stream);

/* Divergence from a teacher that kept K tokens a row:
 *   q = softmax over the kept slots of logits / temperature,
 *   p = softmax over the vocabulary of z / temperature,
 *   loss[t] = sum_k q_k (log q_k - log p[ids_k])
 *   ids     int32 [T,K]  token ids; a negative id marks an empty slot
 *   logits  fp32 [T,K]   the teacher's logits (log-probabilities serve as
 *                        well); -inf marks an empty slot
 *   lse       fp32 [T] out    log-sum-exp of z / temperature
 *   logp_ids  fp32 [T,K] out  log p[ids_k]; -inf in empty slots
 * A row whose slots are all empty is inactive: loss = lse = 0, zero
 * gradient.  The same id in several slots counts as the formulas say: each
 * slot keeps its own log q_k in the loss, which is then below the divergence
 * from the ids' summed q, Q, by sum_k q_k log(Q[ids_k] / q_k), a constant of
 * the teacher (it may be negative); dz has their sum.  A kept slot with an
 * id >= V, or a NaN or +inf logit, makes the row's loss, its grad_h row and
 * grad_W NaN; any finite logits are defined.  1 <= K <= RLK_MAX_K;
 * temperature > 0 and finite (as is its reciprocal). */
rlk_status rlk_linear_distill_fwd(const void* h, const void* W, const int32_t* ids, const float* logits, int64_t T,
                                  int64_t H, int64_t V, int64_t K, float temperature, float* loss, float* lse,
                                  float* logp_ids, void* ws, size_t ws_bytes, void* stream);

/* Gradient of sum_t g[t] loss[t]:
 *   dz_v = (g / temperature) (p_v - sum_{k: ids_k = v} q_k),
 *   grad_h = dz W, grad_W = dz^T h  (outputs as above).
 *   lse, logp_ids  the forward's */
rlk_status rlk_linear_distill_bwd(const void* h, const void* W, const int32_t* ids, const float* logits,
                                  const float* lse, const float* logp_ids, const float* g, int64_t T, int64_t H,
                                  int64_t V, int64_t K, float temperature, void* grad_h, void* grad_W,
                                  int32_t grad_W_dtype, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RLK_VOCAB_OPS_H_ */
