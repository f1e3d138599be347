/*
 * ec_norm.h -- C ABI of the root-mean-square norm in front of a layer on
 * gfx950: with the addition of the residual on the way, its output in its own
 * type or in the 8-bit form of ec_i8.h, and the gradients.
 *
 *   h = x + residual, rounded to x's type (h = x without a residual)
 *   rstd = 1 / sqrt(mean over the row of h^2 + eps)
 *   y = h rstd weight
 *
 * The norm is that of h as it is stored.  Sums and the norm itself are in
 * fp32 (a row whose sum of squares passes fp32's range has rstd = 0), y is
 * rounded once.  `type` is that of x, residual, h, y and their gradients,
 * `wtype` that of weight [cols] and its gradient.
 *
 * Conventions: as in ec_mx.h.  x and the residual have row strides, the other
 * arrays are dense.  Outputs do not overlap inputs.  eps has to be a positive
 * finite number.  Rows are up to EC_MX_MAX_DEPTH elements long.
 */
#ifndef EC_NORM_H
#define EC_NORM_H

#include "ec_mx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* residual and h are both given or both NULL; rstd, f32 [rows], may be NULL. */
ec_status ec_rms_norm(const void* x, uint64_t stride, const void* residual,
                      uint64_t residual_stride, int type, uint64_t rows, uint64_t cols,
                      const void* weight, int wtype, float eps, void* h, void* y, float* rstd,
                      void* stream);

/* The same with y in the 8-bit form, quantized from fp32: codes i8
 * [rows][padded(cols)] (16-byte aligned), scales f32 [rows]. */
ec_status ec_rms_norm_i8(const void* x, uint64_t stride, const void* residual,
                         uint64_t residual_stride, int type, uint64_t rows, uint64_t cols,
                         const void* weight, int wtype, float eps, void* h, void* codes,
                         void* scales, void* stream);

/* Gradients from dy [rows][cols], h and rstd as the forward pass left them, and
 * dh [rows][cols], the gradient that reaches h by other ways (NULL: none):
 *   dx = rstd (weight dy - n mean over the row of weight dy n) + dh, n = h rstd
 *   dweight = sum over the rows of dy n
 * dx is the gradient of x and of the residual alike.  dweight is summed in an
 * order that the sizes fix: in fp32 over runs of up to 256 rows and over what
 * these give to a part, and the parts in 64 bits; with rows = 0 it is zeros.
 * The workspace (16-byte aligned) holds
 * ec_rms_norm_backward_workspace_bytes(rows, cols) bytes. */
size_t ec_rms_norm_backward_workspace_bytes(uint64_t rows, uint64_t cols);
ec_status ec_rms_norm_backward(const void* dy, const void* h, const void* dh, int type,
                               uint64_t rows, uint64_t cols, const float* rstd, const void* weight,
                               int wtype, void* dx, void* dweight, void* workspace,
                               size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EC_NORM_H */
