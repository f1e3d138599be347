/*
 * ec_experts.h -- C ABI of the token exchange of an expert layer on gfx950:
 * tokens sorted by expert (what each rank puts into its all-to-all) and
 * brought back with weights applied, with the gradients of both ways, and a
 * form that sends the tokens in the 4-bit format of ec_mx.h.
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
