/*
 * pop_route.h — C-ABI of routing tokens to experts: scores, a bias for balance, groups of experts,
 * the k best, their weights.
 *
 * For one token with logits l_0 .. l_{E-1} (pop_route_config cfg, an optional bias b):
 *   - expert e is live unless l_e is NaN or -infinity (the marks of a masked expert), or b_e is.
 *     l_e = +infinity counts as the largest finite float.
 *   - scores: POP_ROUTE_SOFTMAX  s_e = exp(l_e - max l) / sum exp(l - max l), over the experts whose l_e is live;
 *             POP_ROUTE_SIGMOID  s_e = 1 / (1 + exp(-l_e)).
 *   - choice values: c_e = s_e + b_e with a bias; without one c_e = s_e (sigmoid) or l_e (softmax: the
 *     same order, without ties that the rounding of s_e would add).
 *   - groups: the experts lie in n_groups runs of E / n_groups. A group's value is the largest c of its
 *     live experts (group_sum 1) or the sum of its two largest (group_sum 2; one if one is live). The
 *     top_groups groups of largest value stay; a group without a live expert never does.
 *   - the top_k live experts of the groups that stay with the largest c, in descending order of c.
 *     Every tie, of experts and of groups, goes to the lower index.
 *   - weights: s_e of the chosen (without the bias); with renorm divided by their sum (all 0 if the sum
 *     is 0); times scale.
 *   - a slot for which no live expert is left gets expert -1 and weight 0.
 * Scores, sums and weights are fp32.
 */
#ifndef POP_ROUTE_H_
#define POP_ROUTE_H_

#include "pop_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define POP_ROUTE_MAX_EXPERTS 256
#define POP_ROUTE_MAX_TOP_K 16

enum { POP_ROUTE_SOFTMAX = 0, POP_ROUTE_SIGMOID = 1 };

typedef struct {
  int n_experts;   /* E, 1..POP_ROUTE_MAX_EXPERTS */
  int top_k;       /* 1..POP_ROUTE_MAX_TOP_K, at most top_groups * E / n_groups */
  int score;       /* POP_ROUTE_SOFTMAX or POP_ROUTE_SIGMOID */
  int n_groups;    /* divides E; 1 = no groups */
  int top_groups;  /* 1..n_groups */
  int group_sum;   /* 1 or 2; 2 needs choice values that are scores: sigmoid, or a bias */
  int renorm;      /* 0 or 1 */
  float scale;     /* finite */
} pop_route_config;

/* Routes T tokens (T >= 0; with 0 only counts is written), on the current device, where all that is given lies.
 *   logits: device [T, E], float32 (logits_bf16 = 0) or bf16 (1), rows ld_logits >= E elements apart,
 *           aligned to its element.
 *   bias:   device float32 [E], or NULL.
 *   experts: device int32 [T, top_k]; weights: device float32 [T, top_k].
 *   counts: device int32 [E], or NULL: receives the number of slots given to each expert (what a bias
 *           for balance is updated from).
 * Asynchronous on `stream`, no allocation; safe to capture in a CUDA graph. One kernel (and one memset
 * with counts). Errors: INVALID_ARG, UNSUPPORTED (not sm_103), CUDA. */
pop_status pop_route(const pop_route_config* cfg, const void* logits, int logits_bf16, long long ld_logits,
                     const float* bias, int T, int* experts, float* weights, int* counts, void* stream);

/* Message of this thread's last failed pop_route. Never NULL. */
const char* pop_route_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* POP_ROUTE_H_ */
