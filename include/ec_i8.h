/*
 * ec_i8.h -- C ABI of the 8-bit integer form on gfx950: rows of whole numbers
 * with one scale each, its inverse, and products of 8-bit operands on the
 * matrix cores, dense and over rows grouped by expert.  It serves the layers
 * of ec_mx.h where four bits are too coarse: weights with a scale for each
 * output channel, activations with a scale for each token.
 *
 * Format ("I8")
 *   - A row has one scale s, f32, and codes, i8: the row's values are s times
 *     its codes.
 *   - With m the row's largest magnitude, s = m / 127 in fp32; a code is the
 *     fp32 quotient x / s rounded to a whole number, ties to even, kept within
 *     [-127, 127].  A row of zeros has s = 0 and codes 0.
 *   - A row that holds a NaN or an infinity has s = NaN and codes 0: all its
 *     values, and all products with it, are NaN.
 *   - A row of c elements is padded with zeros to ec_mx_padded(c) codes: codes
 *     are i8 [rows][padded], scales f32 [rows], both dense.
 *   Codes of a caller's own may be -128 too.
 *
 * Groups and conventions: as in ec_mx.h.  Codes have to be 16-byte aligned,
 * scales 4-byte; padding has to be zero where a product reads it.  Products sum
 * in 32-bit integers, which is exact for every depth that they take; the sum is
 * converted to fp32, multiplied by the row's and then by the column's scale,
 * each rounded to fp32, and then to y's type.
 */
#ifndef EC_I8_H
#define EC_I8_H

#include "ec_mx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Longest contraction of a product (a multiple of 128): 2^14 times this stays
 * below 2^31.  Quantization takes rows of up to EC_MX_MAX_DEPTH. */
#define EC_I8_MAX_DEPTH ((1u << 17) - 128u)

/* Quantize x [rows][cols] (row stride `stride` >= cols) along its rows. */
ec_status ec_i8_quantize(const void* x, int type, uint64_t rows, uint64_t cols, uint64_t stride,
                         void* codes, void* scales, void* stream);

/* y [rows][cols] (row stride `stride`) = scale times code, rounded once more
 * where y's type is shorter than fp32. */
ec_status ec_i8_dequantize(const void* codes, const void* scales, uint64_t rows, uint64_t cols,
                           void* y, int type, uint64_t stride, void* stream);

/* y [rows][cols] = a b^T: a [rows][depth] and b [cols][depth] in the 8-bit
 * form, depth a multiple of 128. */
ec_status ec_i8_product(const void* a_codes, const void* a_scales, uint64_t rows,
                        const void* b_codes, const void* b_scales, uint64_t cols, uint64_t depth,
                        void* y, int type, void* stream);

/* The same in parts of the contraction, where few rows and a long one leave most
 * of the GPU idle: the workspace (16-byte aligned, may be NULL where the size is
 * 0) holds ec_i8_product_parts_bytes(...) bytes, which is 0 where the product is
 * taken in one part, as of more than EC_I8_MOST_PARTS_ROWS rows.  The results are
 * the same. */
#define EC_I8_MOST_PARTS_ROWS 256u
size_t ec_i8_product_parts_bytes(uint64_t rows, uint64_t cols, uint64_t depth);
ec_status ec_i8_product_parts(const void* a_codes, const void* a_scales, uint64_t rows,
                              const void* b_codes, const void* b_scales, uint64_t cols,
                              uint64_t depth, void* y, int type, void* workspace,
                              size_t workspace_bytes, void* stream);

/* y [rows][cols]: row r of group e is a[r] b[e]^T with b [experts][cols][depth];
 * rows of no group are zeros. */
ec_status ec_i8_product_experts(const void* a_codes, const void* a_scales, uint64_t rows,
                                const void* b_codes, const void* b_scales, uint64_t cols,
                                uint64_t depth, const int32_t* offsets, uint32_t experts, void* y,
                                int type, void* stream);

/* What a product of these sizes runs as, where it is taken in one part.
 * ec_i8_product_tile: rows and columns of a tile (256, 128 or 64; 16 where the
 * kernel for few rows runs) in ec_i8_product (experts = 0) or
 * ec_i8_product_experts; 0 if there is no such product.
 * ec_i8_product_rows_first: the rows that ec_i8_product puts into a launch of
 * their own, as tiles of 256, before one for the rest (0: all go in one); each
 * launch's tile is that of its rows. */
uint32_t ec_i8_product_tile(uint64_t rows, uint64_t cols, uint64_t depth, int type,
                            uint32_t experts);
uint64_t ec_i8_product_rows_first(uint64_t rows, uint64_t cols, uint64_t depth, int type);

/* y [rows][cols] = Q(x) w^T: x [rows][depth] is quantized along its rows on
 * the way, w [cols][padded(depth)] is in the 8-bit form.  With experts > 0,
 * rows are grouped by offsets and w is [experts][cols][padded(depth)]; else
 * offsets is NULL.  The workspace (16-byte aligned, may be NULL where the size
 * is 0) holds ec_i8_linear_workspace_bytes(...) bytes. */
size_t ec_i8_linear_workspace_bytes(uint64_t rows, uint64_t depth, uint64_t cols,
                                    uint32_t experts);
ec_status ec_i8_linear(const void* x, int type, uint64_t rows, uint64_t depth, uint64_t stride,
                       const void* w_codes, const void* w_scales, uint64_t cols,
                       const int32_t* offsets, uint32_t experts, void* y, void* workspace,
                       size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EC_I8_H */
