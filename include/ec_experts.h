/*
 * ec_experts.h -- C ABI of the routing and the token exchange of an expert
 * layer on gfx950: experts chosen by their scores, tokens sorted by expert (what
 * each rank puts into its all-to-all) and brought back with weights applied,
 * with the gradients of all of it, and forms that send the tokens in the 4-bit
 * format of ec_mx.h or the 8-bit form of ec_i8.h.
 *
 * A token t has `choices` experts ids[t][j].  An id outside [0, experts) (a
 * router writes -1) is a dropped choice: it takes part in nothing, and what
 * its weight holds has no effect.
 *   - order, i32 [tokens * choices]: row r of the sorted array is the flat
 *     choice order[r] = t * choices + j; choices of one expert keep their
 *     order; rows at offsets[experts] and beyond are -1.
 *   - place, i32 [tokens][choices]: the row of a choice, -1 if dropped.
 *   - offsets, i32 [experts + 1]: expert e owns rows
 *     [offsets[e], offsets[e + 1]).
 * Functions that take a place or an order check each entry against the
 * arrays' sizes on the device: an entry out of range counts as -1.
 *
 * Conventions: as in ec_mx.h.  Rows of x, xs, y, ys and their gradients are
 * dense [.][cols].  Sums run in fp32 in the order of the choices, and results
 * are rounded once.  `wtype` is the type of weights and their gradients.
 */
#ifndef EC_EXPERTS_H
#define EC_EXPERTS_H

#include "ec_mx.h"

#ifdef __cplusplus
extern "C" {
#endif

#define EC_EXPERTS_MAX 1024u
#define EC_EXPERTS_MAX_CHOICES 64u

/* Routing: ids i32 and weights f32 [tokens][choices] of logits [tokens][experts]
 * (row stride `stride`).
 *   - A token's scores are the softmax or the sigmoid of its logits.  Experts
 *     are ordered by score + bias (bias f32 [experts], or NULL: by the logits
 *     themselves), computed in 64 bits, the largest first; a NaN counts as the
 *     largest; of equal ones the lowest index comes first.
 *   - With groups > 1 (dividing experts into runs of as many each), only experts
 *     of the top_groups groups are taken whose two best score + bias sum highest
 *     (of a group with one expert left, that one's).
 *   - An expert whose logit or whose score + bias is -infinity is never taken:
 *     where no other is left, the id is -1 and the weight 0.
 *   - A choice's weight is `scale` times its score, divided by the sum of the
 *     chosen scores with renormalize.  The bias orders only.
 * choices <= experts / groups * top_groups.  EC_ERR_UNSUPPORTED: more than
 * EC_EXPERTS_MAX experts, EC_EXPERTS_MAX_CHOICES choices or
 * EC_EXPERTS_MAX_GROUPS groups. */
typedef enum { EC_SCORE_SOFTMAX = 0, EC_SCORE_SIGMOID = 1 } ec_score;
#define EC_EXPERTS_MAX_GROUPS 64u
ec_status ec_expert_route(const void* logits, int type, uint64_t tokens, uint64_t stride,
                          uint32_t experts, const float* bias, uint32_t choices, int score,
                          uint32_t groups, uint32_t top_groups, int renormalize, float scale,
                          int32_t* ids, float* weights, void* stream);

/* dlogits [tokens][experts] (dense, of the logits' type) from dweights f32
 * [tokens][choices] and the ids of the forward pass; ids outside [0, experts)
 * take no part.  Which experts are chosen has no gradient, nor has the bias. */
ec_status ec_expert_route_backward(const float* dweights, const void* logits, int type,
                                   uint64_t tokens, uint64_t stride, uint32_t experts,
                                   const int32_t* ids, uint32_t choices, int score,
                                   int renormalize, float scale, void* dlogits, void* stream);

/* Bytes of workspace that ec_expert_sort needs (0: none). */
size_t ec_expert_sort_workspace_bytes(uint64_t n, uint32_t experts);

/* Sort n = tokens * choices ids (i32, or i64 with id_bytes = 8) by expert. */
ec_status ec_expert_sort(const void* ids, uint32_t id_bytes, uint64_t n, uint32_t experts,
                         int32_t* order, int32_t* place, int32_t* offsets, void* workspace,
                         size_t workspace_bytes, void* stream);

/* xs [tokens * choices][cols]: xs[place[t][j]] = x[t], zeros in the rows of
 * no expert. */
ec_status ec_expert_dispatch(const void* x, int type, uint64_t tokens, uint64_t cols,
                             const int32_t* place, uint32_t choices, const int32_t* offsets,
                             uint32_t experts, void* xs, void* stream);

/* The same in the 4-bit form: each token is quantized once and its codes and
 * scales are written to its rows (zeros in the rows of no expert). */
ec_status ec_expert_dispatch_mx(const void* x, int type, uint64_t tokens, uint64_t cols,
                                const int32_t* place, uint32_t choices, const int32_t* offsets,
                                uint32_t experts, void* codes, void* scales, void* stream);

/* The dispatch of rows that are in the 8-bit form: x_codes i8 [tokens][padded]
 * (padded a multiple of 128, 16-byte aligned) and x_scales f32 [tokens] to codes
 * [tokens * choices][padded] and scales; rows of no expert hold zeros. */
ec_status ec_expert_dispatch_i8(const void* x_codes, const void* x_scales, uint64_t tokens,
                                uint64_t padded, const int32_t* place, uint32_t choices,
                                const int32_t* offsets, uint32_t experts, void* codes,
                                void* scales, void* stream);

/* Gradient of the dispatch: dx[t] = sum_j dxs[place[t][j]]. */
ec_status ec_expert_dispatch_backward(const void* dxs, int type, uint64_t tokens, uint64_t cols,
                                      const int32_t* place, uint32_t choices, void* dx,
                                      void* stream);

/* y[t] = sum_j weights[t][j] ys[place[t][j]]. */
ec_status ec_expert_combine(const void* ys, int type, uint64_t tokens, uint64_t cols,
                            const int32_t* place, uint32_t choices, const void* weights,
                            int wtype, void* y, void* stream);

/* Its gradients: dys[place[t][j]] = weights[t][j] dy[t] (zeros in the rows of
 * no expert), dweights[t][j] = <dy[t], ys[place[t][j]]> (0 if dropped). */
ec_status ec_expert_combine_backward(const void* dy, const void* ys, int type, uint64_t tokens,
                                     uint64_t cols, const int32_t* place, uint32_t choices,
                                     const void* weights, int wtype, const int32_t* offsets,
                                     uint32_t experts, void* dys, void* dweights, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EC_EXPERTS_H */
