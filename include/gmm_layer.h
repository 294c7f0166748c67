/*
 * gmm_layer.h -- both ends of a mixture-of-experts layer, in libgmm.so beside
 * the grouped matmul (gmm.h) and the token operators (gmm_moe.h): the router
 * (its choice of experts, the balance loss with per-expert counts, and the
 * gradient of both), the experts' products of a few tokens by expert id over
 * four-bit weights, and the AdamW step of many tensors.
 *
 * A layer's training step is
 *
 *   gmm_route_run         logits [T,E]     -> expert ids and weights [T,k]
 *   gmm_balance_loss_run  logits, ids      -> loss, counts [E], tokens
 *   (gmm_moe.h, gmm.h)    sort, dispatch, products, combine, their gradients
 *   gmm_router_grad_run   dweights, counts -> dlogits [T,E]
 *   gmm_adamw_run         gradients        -> weights, states
 *
 * and a decode step of a few tokens gmm_route_run, then gmm_gmv_run for each
 * projection: no sort, no expert rows.
 *
 * The conventions of gmm.h hold: dense row-major device tensors that the
 * caller owns, 16-byte aligned; every call only queues work on `stream`,
 * allocates nothing and can be captured into a graph; a gmm_status comes
 * back, with a text from gmm_last_error; a refused call queues nothing.
 * Outputs must not overlap inputs or each other (GMM_E_INVALID).  Workspaces
 * need no preparation and are of no use afterwards; two calls that may overlap
 * in time need one each.  All sums have a fixed order: equal inputs give equal
 * bits.
 */
#ifndef GMM_MI355X_GMM_LAYER_H
#define GMM_MI355X_GMM_LAYER_H

#include <stddef.h>

#include "gmm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How a router's logits z become scores s: a softmax over the experts, or a
 * sigmoid of each. */
#define GMM_SCORES_SOFTMAX 0
#define GMM_SCORES_SIGMOID 1

/*
 * The router's tensors, in all three of its calls:
 *
 *   logits      [T,E] F32 or BF16; everything is computed in fp32.  An expert
 *               whose logit is -inf is switched off for its token.
 *   valid       NULL, or [T] I8: a token with 0 here is padding, and its
 *               logits are not read into anything, whatever they hold.
 *   expert_ids  [T,k] I32 (written by gmm_route_run), I32 or I64 (read by the
 *               others).  When read, an id outside [0,E) is no choice, and the
 *               same expert may appear twice in a token.
 *
 * Scores below 2^-126 may count as 0.
 *
 * A token counts when it is valid and has an expert that is not switched off.
 * A NaN or +inf logit of a token that counts makes what depends on it NaN.
 * Limits: 1 <= E <= 1024, 1 <= k <= 64, k <= E, T*E < 2^31 (GMM_E_UNSUPPORTED
 * above, GMM_E_INVALID for k > E).
 */

/*
 * gmm_route_run: queue the choice of k experts for every token:
 *   those with the largest logits -- with a bias, the largest s + bias (one
 *   fp32 addition) -- equal ones in the order of their ids, the best first;
 *   weights[t,j] = scale * s_j / S, with s the score of choice j (the bias is
 *   no part of it) and S the sum of the token's chosen scores with
 *   renormalize, else 1 (and 0 where S is 0).
 * An expert that is switched off is never chosen: a token that has fewer than
 * k others gets ids -1 and weights 0 behind them, and so does a token that
 * does not count.  A token with a NaN or +inf logit gets ids -1 and weights NaN.
 *
 *   bias        NULL or [E] F32.  An expert whose bias is -inf is never chosen
 *               (its score still counts in the softmax); a NaN or +inf of s +
 *               bias acts as one of a logit.
 *   expert_ids  [T,k] I32, written.
 *   weights     [T,k] F32, written.
 */
gmm_status gmm_route_run(gmm_handle* h,
                         const gmm_tensor* logits,
                         const gmm_tensor* bias,
                         const gmm_tensor* valid,
                         int scores,
                         int renormalize,
                         float scale,
                         const gmm_tensor* expert_ids,
                         const gmm_tensor* weights,
                         void* stream);

/*
 * gmm_balance_loss_workspace: bytes of workspace that gmm_balance_loss_run
 * needs for T tokens and E experts (0 for a few tokens).
 */
gmm_status gmm_balance_loss_workspace(int64_t tokens, int64_t experts, size_t* bytes);

/*
 * gmm_balance_loss_run: queue, over the n tokens that count,
 *   counts[e] = choices of expert e (of any token),
 *   p[t,e]    = s[t,e] / sum over e of s[t,e] (0 where that sum is 0),
 *   loss      = coef * E * sum over e of f[e] * P[e]
 *               + z_coef * mean over t of logsumexp(z[t])^2,
 * with f[e] = counts[e] / max(1, sum of counts) and P[e] the mean of p[t,e]
 * over t (0 when n = 0).
 *
 *   loss     [1] F32, written.
 *   counts   [E] I32, written.
 *   tokens   [1] I32, written: n.
 */
gmm_status gmm_balance_loss_run(gmm_handle* h,
                                const gmm_tensor* logits,
                                const gmm_tensor* expert_ids,
                                const gmm_tensor* valid,
                                int scores,
                                float coef,
                                float z_coef,
                                const gmm_tensor* loss,
                                const gmm_tensor* counts,
                                const gmm_tensor* tokens,
                                void* workspace,
                                size_t workspace_bytes,
                                void* stream);

/*
 * gmm_router_grad_run: queue the gradient with respect to the logits of
 *   sum over t,j of dweights[t,j] * weights[t,j]   (gmm_route_run's weights
 *                                                   for these expert_ids), and
 *   dloss * loss                                   (gmm_balance_loss_run's),
 * the counts being constants.  Either part may be left out: dweights NULL, or
 * counts and tokens NULL.  Counts and tokens may also be sums over the ranks
 * of a data-parallel job (the loss is then that of the whole batch).  Tokens
 * that do not count get zeros, and so do experts that are switched off.
 *
 *   dweights  NULL or [T,k] F32 or BF16; not read where there is no choice.
 *   counts    NULL or [E] I32, tokens [1] I32, as gmm_balance_loss_run writes
 *             them.
 *   dloss     NULL (1) or [1] F32.
 *   dlogits   [T,E], logits' type, written.
 */
gmm_status gmm_router_grad_run(gmm_handle* h,
                               const gmm_tensor* logits,
                               const gmm_tensor* expert_ids,
                               const gmm_tensor* valid,
                               int scores,
                               const gmm_tensor* dweights,
                               int renormalize,
                               float scale,
                               const gmm_tensor* counts,
                               const gmm_tensor* tokens,
                               const gmm_tensor* dloss,
                               float coef,
                               float z_coef,
                               const gmm_tensor* dlogits,
                               void* stream);

/*
 * gmm_gmv_workspace: bytes of workspace that gmm_gmv_run needs for a product
 * of `slots` = T*k rows to N columns (0 without weights, and for a few slots).
 */
gmm_status gmm_gmv_workspace(int64_t slots, int64_t N, int weighted, size_t* bytes);

/*
 * gmm_gmv_run: queue the products of a few tokens with the weights of their
 * experts, by expert id (no sorting, no expert rows):
 *   y[t,j,n] = sum over k of W(id[t,j], n, k) * x[t,k]      (x [T,K]) or
 *              sum over k of W(id[t,j], n, k) * x[t,j,k]    (x [T,k,K]),
 *   W(g,n,k) = rhs_scale[g,b,0,n] * (rhs[g,n,k] - rhs_zero[g,b,0,n]),
 * b being k's block of K/nb elements.  Without weights out = y; with them
 * out[t] = sum over j of weights[t,j] * y[t,j].  The weights and scales are
 * gmm_run's own (rhs_format, rhs_scale), so a larger batch goes there with the
 * same tensors.  Products and sums are fp32, rounded once.  A slot whose id is
 * outside [0,G) gives zeros: its x and weight are not read into anything.
 *
 * With I4 and U4 codes times x and sums of x are added apart, and I4 codes as
 * code + 8 (with or without zero points): the roundings, each 2^-24 of a partial
 * sum, go by |scale| (|code| + |zero| + 16) |x| (U4: without the 16).  An
 * infinity in a slot's x gives that slot NaN where the formula has an infinity,
 * and so do finite x whose sums of (|code| + 8) |x| or (|zero| + 8) |x| pass
 * fp32's range.
 *
 * F4E2M1 weights with E8M0 scales are widened to bf16 together, as in gmm_run:
 * exact for bytes 0 .. 252; weights past the largest bf16 (bytes 253 and 254)
 * become infinities; byte 255 makes its block NaN.
 *
 *   x           [T,K] or [T,k,K] BF16.
 *   rhs         [G,N,K] I4, U4 or F4E2M1 (two to a byte), K % 32 == 0.
 *   rhs_scale   [G,nb,1,N] F32 or BF16, or with F4E2M1 E8M0 (nb = K/32);
 *               K/nb a multiple of 32.
 *   rhs_zero    NULL (0) or of rhs_scale's shape and type, with I4 and U4.
 *   expert_ids  [T,k] I32 or I64, or NULL with G = 1 (k = 1, every id 0).
 *   weights     NULL or [T,k], F32 or BF16.
 *   out         [T,k,N], with weights [T,N]; F32 or BF16.
 * Limits: T*k <= 4096, 1 <= k <= 64, G <= 1024, N < 2^24, K < 2^20
 * (GMM_E_UNSUPPORTED above).  The time grows with the rows an expert has, every
 * sixteen reading its weight again: from some 16 rows an expert on (a single
 * expert: 80) sorted rows and gmm_run are faster, also within the limit.
 */
gmm_status gmm_gmv_run(gmm_handle* h,
                       const gmm_tensor* x,
                       const gmm_tensor* rhs,
                       const gmm_tensor* rhs_scale,
                       const gmm_tensor* rhs_zero,
                       const gmm_tensor* expert_ids,
                       const gmm_tensor* weights,
                       const gmm_tensor* out,
                       void* workspace,
                       size_t workspace_bytes,
                       void* stream);

/* Elements of an eight-bit state that share a scale. */
#define GMM_ADAMW_BLOCK 256

/* One tensor of a step: n elements, and where they are. */
typedef struct {
  int64_t n;
  void* param;              /* F32 or BF16, read and written */
  const void* grad;         /* F32 or BF16 */
  void* exp_avg;            /* F32, or eight-bit: F8E4M3FN codes; read and written */
  void* exp_avg_sq;         /* the same */
  float* exp_avg_scale;     /* eight-bit states: ceil(n/256) scales, read and written; else NULL */
  float* exp_avg_sq_scale;  /* the same */
  void* copy;               /* NULL, or BF16: the parameter rounded, written */
} gmm_adamw_item;

typedef struct {
  int32_t param_dtype, grad_dtype; /* GMM_F32 or GMM_BF16 */
  int32_t state_dtype;             /* GMM_F32 or GMM_F8E4M3FN */
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;                    /* of this call, from 1 */
  const int32_t* step_at;          /* NULL, or the step in device memory (a graph's replays) */
  const float* lr_at;              /* NULL, or the learning rate in device memory */
  const float* grad_scale;         /* NULL, or a factor of every gradient in device memory */
} gmm_adamw_args;

/*
 * gmm_adamw_run: queue one AdamW step (decoupled weight decay) of `count`
 * tensors.  Per element, in fp32, every operation rounded to nearest and in
 * this order:
 *   g  = grad * grad_scale
 *   m  = beta1 * m + (1 - beta1) * g
 *   v  = beta2 * v + (1 - beta2) * (g * g)
 *   p  = p * (1 - lr * weight_decay)
 *        - lr / (1 - beta1^step) * (m / (sqrt(v) * 1 / sqrt(1 - beta2^step) + eps))
 * the factors that do not depend on the element being computed in double and
 * rounded once.  A bf16 parameter is rounded to nearest at the end; `copy`
 * takes that rounding of an fp32 one (the weights that the products read).
 *
 * Eight-bit states hold e4m3fn codes and one fp32 scale per block of 256
 * consecutive elements of a tensor (the last one may be short): m is
 * code * scale, and v the square of code * scale (codes of sqrt(v)).  After
 * the step, scale = max(amax * c, 2^-126) of the block, c being 1/448 rounded
 * to fp32 (448 is the largest code's value; 1 when all are zero), code = the
 * value nearest to x / scale, ties to the even code, and for sqrt(v) at least
 * the smallest code above zero where v > 0.  A block
 * that holds an infinity or a NaN gets a NaN scale and zero codes.
 *
 * The tensors of a step must not overlap, and a tensor has fewer than 2^34
 * elements (GMM_E_UNSUPPORTED from there on).  With step_at, a step below 1 counts
 * as 1.
 *
 * A step of many tensors is several launches: when one of them fails
 * (GMM_E_HIP), those before it stay queued, and the call must not be repeated
 * as it is.
 */
gmm_status gmm_adamw_run(gmm_handle* h,
                         const gmm_adamw_item* items,
                         int64_t count,
                         const gmm_adamw_args* args,
                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GMM_MI355X_GMM_LAYER_H */
