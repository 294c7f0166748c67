/*
 * gmm_moe.h -- the steps around the grouped matmul of a mixture-of-experts
 * layer, in libgmm.so beside it (gmm.h): tokens sorted by expert, dispatched
 * into expert rows and combined back with their router weights, the gradients
 * of both, and microscaled fp4 tensors (blocks of 32 elements of K with one
 * E8M0 scale), quantised and widened.
 *
 * Notation: T tokens of D columns, k choices each; n = T*k slots, slot (t,j)
 * being number t*k + j; G experts.  A layer's forward pass is
 *
 *   gmm_sort_tokens_run   expert ids [T,k] -> group_sizes [G], slot_row [T,k]
 *   gmm_dispatch_run      x [T,D]          -> rows [n,D], sorted by expert
 *   gmm_run ...           rows             -> expert outputs [n,D']
 *   gmm_combine_run       expert outputs   -> out [T,D']
 *
 * and its backward pass gmm_combine_grad_run, the gmm and tgmm gradients, and
 * gmm_combine_run without weights, which is the gradient of gmm_dispatch_run.
 *
 * The conventions of gmm.h hold: dense row-major device tensors that the
 * caller owns, 16-byte aligned; every call only queues work on `stream`,
 * allocates nothing and can be captured into a graph; a gmm_status comes
 * back, with a text from gmm_last_error; a refused call queues nothing.
 * Outputs must not overlap inputs or each other (GMM_E_INVALID).
 */
#ifndef GMM_MI355X_GMM_MOE_H
#define GMM_MI355X_GMM_MOE_H

#include <stddef.h>

#include "gmm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Reported by gmm_device_flags: a slot_row entry named a row outside
 * [0, T*k) (as itself or as a complement).  Its slot counted as unrouted and
 * wrote no row. */
#define GMM_FLAG_BAD_ROW 0x10u

/*
 * gmm_sort_tokens_workspace: bytes of workspace that gmm_sort_tokens_run
 * needs for `slots` = T*k slots and `groups` = G experts (0 for a sort that
 * one workgroup does).  GMM_E_INVALID for a negative count or a NULL bytes,
 * GMM_E_UNSUPPORTED outside gmm_sort_tokens_run's limits.
 */
gmm_status gmm_sort_tokens_workspace(int64_t slots, int64_t groups, size_t* bytes);

/*
 * gmm_sort_tokens_run: queue the stable sort of T*k slots by expert.
 *
 *   expert_ids   [T,k] I32 or I64.  An id outside [0,G) (a dropped slot, or
 *                an expert of another shard) leaves its slot unrouted.  The
 *                same expert may appear twice in a token.
 *   group_sizes  [G] I32, written: the slots of each expert (what gmm takes).
 *   slot_row     [T,k] I32, written: the slot's row in the sorted order,
 *                slots of one expert in slot order.  Unrouted slots come
 *                after all others, in slot order; they hold the bitwise
 *                complement of their row (a negative number), so slots and
 *                rows 0..T*k-1 correspond one to one.
 *   workspace    device memory of at least gmm_sort_tokens_workspace bytes,
 *                16-byte aligned (NULL when that is 0).  Its contents need
 *                no preparation and are of no use afterwards; two calls that
 *                may overlap in time need a workspace each.
 *
 * Limits: 1 <= G <= 1024, 1 <= k <= 64, T*k < 2^31 (GMM_E_UNSUPPORTED above).
 */
gmm_status gmm_sort_tokens_run(gmm_handle* h,
                               const gmm_tensor* expert_ids,
                               const gmm_tensor* group_sizes,
                               const gmm_tensor* slot_row,
                               void* workspace,
                               size_t workspace_bytes,
                               void* stream);

/*
 * gmm_dispatch_run: queue the copy of every token to its expert rows:
 * out[slot_row[t,j]] = x[t].  The rows of unrouted slots (the tail rows that
 * slot_row names by complements) are filled with zeros, so all T*k rows are
 * written.
 *
 *   x         [T,D], any one-, two- or four-byte type (values are copied as
 *             they are, so scales [T,K/128] or quantised rows go the same way).
 *   slot_row  [T,k] I32, as gmm_sort_tokens_run writes it.
 *   out       [T*k,D], x's type.
 * Limits: 1 <= k <= 64, T*k < 2^31, D < 2^28 (GMM_E_UNSUPPORTED above).
 */
gmm_status gmm_dispatch_run(gmm_handle* h,
                            const gmm_tensor* x,
                            const gmm_tensor* slot_row,
                            const gmm_tensor* out,
                            void* stream);

/*
 * gmm_combine_run: queue out[t] = sum over routed slots (t,j) of
 * weights[t,j] * rows[slot_row[t,j]], in fp32 in the order of j, rounded once
 * to the output type.  Without weights (NULL) every weight is 1: the gradient
 * of gmm_dispatch_run.  The rows and weights of unrouted slots are not read
 * into the sum, whatever they hold; a token without a routed slot gets zeros.
 *
 *   rows      [T*k,D] F32 or BF16.
 *   slot_row  [T,k] I32.
 *   weights   NULL or [T,k], F32 or BF16.
 *   out       [T,D] F32 or BF16.
 * Limits as for gmm_dispatch_run.
 */
gmm_status gmm_combine_run(gmm_handle* h,
                           const gmm_tensor* rows,
                           const gmm_tensor* slot_row,
                           const gmm_tensor* weights,
                           const gmm_tensor* out,
                           void* stream);

/*
 * gmm_combine_grad_run: queue the gradients of gmm_combine_run with weights:
 *   drows[slot_row[t,j]] = weights[t,j] * dout[t]        (zeros in the rows of
 *                                                         unrouted slots),
 *   dweights[t,j] = sum over d of dout[t,d] * rows[slot_row[t,j],d]
 *                                                        (0 when unrouted),
 * in fp32, each rounded once to its type.  The sums are taken in a fixed
 * order: equal inputs give equal bits.
 *
 *   dout      [T,D] F32 or BF16.
 *   rows      [T*k,D] F32 or BF16, the rows that gmm_combine_run read.
 *   slot_row  [T,k] I32.
 *   weights   [T,k] F32 or BF16.
 *   drows     [T*k,D], rows' type; every row is written.
 *   dweights  [T,k], weights' type.
 * Limits as for gmm_dispatch_run.
 */
gmm_status gmm_combine_grad_run(gmm_handle* h,
                                const gmm_tensor* dout,
                                const gmm_tensor* rows,
                                const gmm_tensor* slot_row,
                                const gmm_tensor* weights,
                                const gmm_tensor* drows,
                                const gmm_tensor* dweights,
                                void* stream);

/*
 * gmm_quant_mxfp4_run: queue the quantisation of x to fp4 e2m1 in blocks of
 * 32 consecutive elements of K, each with an E8M0 scale:
 *   E    = floor(log2(amax of the block)) - 2, clamped to [-127, 125]
 *          (0 for an all-zero block),
 *   byte = E + 127,
 *   code = the e2m1 value nearest to x * 2^-E, ties to the even code, the
 *          sign kept, magnitudes beyond 6 taken as 6.
 * A block that holds an infinity or a NaN gets byte 255 (NaN in the
 * microscaling encoding) and zero codes.
 *
 *   x      [M,K] or [Ga,N,K], BF16 or F32, K % 32 == 0.
 *   q      F4E2M1 of x's shape (two codes a byte, the even element in the low
 *          nibble), written.
 *   scale  E8M0, written: for x [M,K] the layout of gmm_run's lhs_scale,
 *          [M,K/32]; for x [Ga,N,K] that of its rhs_scale, [Ga,K/32,1,N].
 * Limits: M, or Ga*N, below 2^31 and K below 2^28 (GMM_E_UNSUPPORTED above).
 */
gmm_status gmm_quant_mxfp4_run(gmm_handle* h,
                               const gmm_tensor* x,
                               const gmm_tensor* q,
                               const gmm_tensor* scale,
                               void* stream);

/*
 * gmm_widen_mxfp4_run: queue the values that q and scale stand for:
 * y = value(code) * 2^(byte - 127), exact in F32 and in BF16 (a value past
 * either type's largest becomes an infinity); every element of a block with
 * byte 255 is NaN.
 *   q, scale  as gmm_quant_mxfp4_run writes them.
 *   y         BF16 or F32 of q's shape, written.
 */
gmm_status gmm_widen_mxfp4_run(gmm_handle* h,
                               const gmm_tensor* q,
                               const gmm_tensor* scale,
                               const gmm_tensor* y,
                               void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GMM_MI355X_GMM_MOE_H */
