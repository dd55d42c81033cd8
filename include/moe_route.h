/*
 * moe_route.h — C ABI of routing beyond the layer's own softmax top-k (one GB300
 * GPU, sm_103a): softmax or sigmoid scores, a bias for balance, groups of
 * experts, renormalised weights; and the layer call that takes such a choice.
 *
 * The conventions are those of moe_attention.h: a return code per call, device
 * pointers owned by the caller, work stream-ordered on the caller's stream, no
 * allocation, no host synchronisation, capturable; moe_route has no handle and may
 * be called from several threads and streams at once.
 */
#ifndef MOE_ROUTE_H
#define MOE_ROUTE_H

#include "moe_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1
#define MOE_GROUP_MAX 0  /* a group is worth its largest value                 */
#define MOE_GROUP_TOP2 1 /* a group is worth the sum of its two largest values */

#define MOE_ROUTE_BAD_LOGIT 16 /* status bit: a logit was NaN or +infinity, or the bias not finite */

typedef struct {
  int32_t n_experts;   /* E, 1..1024                                                  */
  int32_t top_k;       /* k, 1..32, at most the experts of the kept groups            */
  int32_t score;       /* MOE_SCORE_*                                                 */
  int32_t n_groups;    /* 1..32, E a multiple of it; group g is the experts
                          [g E / n_groups, (g + 1) E / n_groups)                      */
  int32_t top_groups;  /* groups that experts are chosen from, 1..n_groups            */
  int32_t group_score; /* MOE_GROUP_*                                                 */
  int32_t renormalise; /* weights sum to `scale`                                      */
  float scale;         /* finite; of every weight                                     */
} moe_routing;

/*
 * The experts of n_tokens tokens and their weights.
 * Scores p = softmax(x) or 1 / (1 + exp(-x)) of a token's logits x; values c = p +
 * bias (fp32 [E], or NULL: then experts are taken in the order of their logits).
 * The top_groups groups of largest worth are kept (ties: the lower group), and of
 * their experts the top_k of largest c are chosen, in descending order (ties: the
 * lower expert).  weights = scale p of the chosen, divided by the chosen's sum of p
 * where renormalise is not 0.  The choice is that of values formed in 64 bits.
 * A logit of -infinity closes an expert: it comes after all others, with weight 0,
 * and adds nothing to its group's worth (a group of none but such comes last).
 * A row with a NaN or +infinity, or with a bias that is not finite, gives the
 * experts 0..k-1 with weights NaN, and a status.
 * logits: [n_tokens][E] in dtype (MOE_F32, MOE_BF16, MOE_F16), rows token_stride
 * elements apart.  ids int32, weights fp32: [n_tokens][top_k] contiguous.
 * status: device word, or NULL.
 */
int moe_route(const moe_routing *r, const void *logits, int64_t token_stride, int32_t n_tokens, const float *bias,
              int32_t *ids, float *weights, int32_t dtype, int32_t *status, void *cuda_stream);

/*
 * moe_layer_forward with the choice made by the caller: d_ids int32 and d_weights
 * fp32, device [n_tokens][top_k] contiguous, in place of logits.  The weights are
 * used as they are.  A token's experts are distinct and in [0, n_experts), and its
 * weights finite; what is not so is an error like a non-finite logit's.
 */
int moe_layer_forward_routed(moe_cache *c, int32_t layer, const int32_t *d_ids, const float *d_weights, const void *d_x,
                             int32_t n_tokens, float *d_out, void *cuda_stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_ROUTE_H */
