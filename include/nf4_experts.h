/*
 * nf4_experts.h -- C ABI of what stands around the grouped products of libnf4.so:
 * a router's choice of experts with the order in which the grouped calls of
 * nf4.h and nf4_int8.h take the rows, the tokens' rows to their experts'
 * places, and the experts' rows back to their tokens.  Each with its backward
 * pass.
 *
 * Conventions (memory, streams, errors, status codes) are those of nf4.h: all
 * pointers are device memory of the caller, work is enqueued asynchronously
 * on `stream`, nothing is allocated, freed or retained, an error enqueues
 * nothing.  Sums run in a fixed order (the only atomics count integers),
 * so repeated calls on the same inputs give bitwise identical outputs.
 * Every call can be captured into a HIP graph.  Written tensors are contiguous
 * and overlap nothing that the call reads.
 *
 * Sizes.  T tokens, E experts (1 to 1024), k choices per token (1 to 64, at
 * most E; of a choice made elsewhere, which may name an expert twice, also more).
 * T * k is at most 2^30, a row has at most 2^23 elements, and a launch holds fewer
 * than 2^32 threads (else NF4_ERR_UNSUPPORTED).  dtype is NF4_DTYPE_F32 or
 * NF4_DTYPE_BF16.
 *
 * The plan of a choice `experts` int32 [T, k]:
 *   offsets  int32 [E + 1]  rows offsets[e] .. offsets[e+1]-1 are expert e's, as
 *                           the grouped calls take them; inside an expert they
 *                           stand in the order of the tokens (t, then j)
 *   tokens   int32 [T * k]  the token whose row stands there; -1 in the rows
 *                           behind offsets[E]
 *   slots    int32 [T, k]   the row of each choice; -1 where there is none
 * An entry of `experts` outside 0 .. E-1 (such as -1) is no choice: it has no
 * row, and the rows that remain behind offsets[E] belong to nobody.  An expert
 * named twice by one token gets two rows.
 */
#ifndef NF4_EXPERTS_H_
#define NF4_EXPERTS_H_

#include "nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define NF4_SCORE_SOFTMAX 0
#define NF4_SCORE_SIGMOID 1

#define NF4_GROUP_MAX  0  /* a group is as good as its best expert           */
#define NF4_GROUP_TOP2 1  /* a group is as good as its best two together     */

/*
 * nf4_route_fwd -- the k experts of each token and their weights.
 *   logits   [T, E] in dtype, rows `stride` elements apart
 *   s        softmax over the E logits of the token, or the sigmoid of each
 *   order    by s, where bias (f32 [E], or NULL) is given by c = s + bias, computed and
 *            compared in 64 bits; equal ones by index.  The bias moves the
 *            choice, never a weight.  Without a bias the order is that of the logits.
 *   groups   the experts in `groups` equal runs, of which only the top_groups
 *            best take part (NF4_GROUP_*: the largest c, or the sum of the two
 *            largest in 64 bits; equal ones by index); 1 and 1 for none
 *   weights  f32 [T, k]: scale * s of the chosen, with renormalize divided by
 *            their sum; scale is positive and finite
 *   experts  int32 [T, k], best first
 *   offsets, tokens, slots: the plan of the choice, or all NULL
 * An expert whose logit is minus infinity (or whose c is) is never chosen: a
 * token that has fewer than k others gets -1 and weight 0 in the remaining
 * places.  A NaN orders before every number, and the weights it reaches are NaN.
 *   ws       nf4_expert_plan_workspace(T, k, E) bytes, 16-byte aligned (none
 *            without a plan)
 */
int nf4_route_fwd(const void* logits, int dtype, int64_t stride, int64_t T, int32_t E,
                  int32_t k, const float* bias, int score, int32_t groups,
                  int32_t top_groups, int group_score, int renormalize, float scale,
                  float* weights, int32_t* experts, int32_t* offsets,
                  int32_t* tokens, int32_t* slots, void* ws, size_t ws_bytes,
                  void* stream);

/*
 * nf4_route_bwd -- grad_logits [T, E] in dtype from grad_weights f32 [T, k] and
 * the forward call's logits, weights and experts (none twice for a token).  The
 * choice itself has no gradient; grad_weights in places without an expert is not read into it.
 */
int nf4_route_bwd(const float* grad_weights, const void* logits, int dtype,
                  int64_t stride, int64_t T, int32_t E, int32_t k, const float* weights,
                  const int32_t* experts, int score, int renormalize, float scale,
                  void* grad_logits, void* stream);

/* nf4_expert_plan -- the plan of a choice made elsewhere. */
int nf4_expert_plan(const int32_t* experts, int64_t T, int32_t k, int32_t E,
                    int32_t* offsets, int32_t* tokens, int32_t* slots, void* ws,
                    size_t ws_bytes, void* stream);

/* Workspace bytes of nf4_expert_plan and of nf4_route_fwd with a plan; SIZE_MAX for
 * sizes they refuse.  A workspace belongs to one call at a time: calls that may
 * overlap (other streams, graphs replayed side by side) take different ones. */
size_t nf4_expert_plan_workspace(int64_t T, int32_t k, int32_t E);

/*
 * nf4_expert_gather -- rows [T * k, H]: row slots[t, j] = x[t].  x [T, H] in
 * dtype, rows `stride` elements apart.  `end` points at one int32, offsets[E] of the
 * plan: the rows behind it are written as zeros where fill_outside is 1, and
 * left as they were where it is 0.
 */
int nf4_expert_gather(const void* x, int dtype, int64_t stride, int64_t T, int64_t H,
                      int32_t k, const int32_t* slots, const int32_t* end, void* rows,
                      int fill_outside, void* stream);

/* nf4_expert_gather_bwd -- grad_x [T, H]: grad_x[t] = sum over j of
 * grad_rows[slots[t, j]], summed in fp32 and rounded once; zeros without any. */
int nf4_expert_gather_bwd(const void* grad_rows, int dtype, int64_t T, int64_t H,
                          int32_t k, const int32_t* slots, void* grad_x, void* stream);

/*
 * nf4_expert_combine_fwd -- out [T, H]: out[t] = sum over j of weights[t, j] *
 * rows[slots[t, j]], in the order of j, summed in fp32 and rounded once.  A choice
 * without a row adds nothing, whatever its weight.
 */
int nf4_expert_combine_fwd(const void* rows, int dtype, int64_t T, int64_t H, int32_t k,
                           const float* weights, const int32_t* slots, void* out,
                           void* stream);

/*
 * nf4_expert_combine_bwd -- from grad_out [T, H] (rows grad_stride elements
 * apart): grad_rows [T * k, H], row slots[t, j] = weights[t, j] * grad_out[t] (NULL if
 * not wanted; rows behind *end by fill_outside as above), and grad_weights f32
 * [T, k] = grad_out[t] . rows[slots[t, j]], 0 without a row (NULL if not wanted; rows
 * may then be NULL).
 */
int nf4_expert_combine_bwd(const void* grad_out, int64_t grad_stride, const void* rows,
                           int dtype, int64_t T, int64_t H, int32_t k,
                           const float* weights, const int32_t* slots,
                           const int32_t* end, void* grad_rows, float* grad_weights,
                           int fill_outside, void* stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* NF4_EXPERTS_H_ */
