/*
 * ec_mx.h -- C ABI of the microscaled 4-bit floating-point format on gfx950:
 * quantization, its inverse, and products of 4-bit operands on the matrix
 * cores (dense, over rows grouped by expert, and per expert over tokens).
 * It serves the layers whose activations and gradients cross the all-to-all
 * of an expert-parallel model, as ec.h serves embedding traffic.
 *
 * Format ("MX4": E2M1 elements with E8M0 block scales)
 *   - 32 consecutive elements of a row (a block) share a scale 2^(s - 127),
 *     held as the byte s.  s = 255 marks a block that held a NaN or an
 *     infinity; all its values read as NaN.
 *   - An element is a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6, as a 4-bit
 *     code (sign in bit 3); the even element of a pair is the low half of
 *     its byte.
 *   - With m the block's largest magnitude, s = max(0, floor(log2 m) + 125);
 *     elements are x / 2^(s - 127) rounded to the nearest value, ties to the
 *     even code, saturating at 6.  A block of zeros has s = 0.
 *   - A row of c elements is padded with zeros to ec_mx_padded(c) = c rounded
 *     up to 128: codes are u8 [rows][padded / 2], scales u8
 *     [rows][padded / 32], both dense.
 *
 * Groups: rows of an array sorted by expert, described by offsets, i32
 * [groups + 1] in device memory: group g is rows [offsets[g], offsets[g+1]).
 * Offsets have to increase (not strictly) from 0; rows at offsets[groups] and
 * beyond belong to no group, and products write zeros there.  They are not
 * checked on the host: values out of order or range give wrong rows but no
 * access outside the arrays.
 *
 * Conventions: as in ec.h (status codes, stream handles, caller-owned device
 * memory; calls enqueue kernels and never allocate or synchronize, so they
 * can be captured into graphs).  Inputs and outputs x, y need the alignment
 * of their element; codes have to be 16-byte aligned, scales that are written
 * 16-byte and scales that are read 4-byte aligned: any rows of a tensor, in
 * a row, are a tensor to read.  Strides are in elements.  Results do not depend on the run: no sum's order is left
 * to chance.
 */
#ifndef EC_MX_H
#define EC_MX_H

#include "ec.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { EC_TYPE_F32 = 0, EC_TYPE_F16 = 1, EC_TYPE_BF16 = 2 } ec_type;

#define EC_MX_BLOCK 32u
/* Longest row (elements, padded, without what groups add to it), most groups,
 * and most rows of one call. Calls of more than 2^31 - 1 workgroups (a
 * quantization of 64 rows of up to 128 elements is one) are
 * EC_ERR_UNSUPPORTED too. */
#define EC_MX_MAX_DEPTH (1u << 24)
#define EC_MX_MAX_GROUPS 1024u
#define EC_MX_MAX_ROWS 0x7fffff00u

/* cols rounded up to a multiple of 128. */
uint64_t ec_mx_padded(uint64_t cols);

/* Padded length of a transposed row over grouped tokens: every group starts
 * at a multiple of 128, so up to 127 elements a nonempty group are added. */
uint64_t ec_mx_padded_groups(uint64_t rows, uint32_t groups);

/* Quantize x [rows][cols] (row stride `stride` >= cols) along its rows.
 * EC_ERR_INVALID: NULL or misaligned pointers, an unknown type, cols = 0, a
 * short stride; EC_ERR_UNSUPPORTED: beyond the limits above.  rows = 0 is a
 * call without work (for every function here). */
ec_status ec_mx_quantize(const void* x, int type, uint64_t rows, uint64_t cols, uint64_t stride,
                         void* codes, void* scales, void* stream);

/* Quantize x [batch][rows][cols] along its rows (row_codes
 * [batch * rows][padded(cols) / 2], row_scales) and along its columns
 * (col_codes [batch * cols][padded(rows) / 2], col_scales), reading x once.
 * Both pointers of one direction may be NULL: that direction is left out. */
ec_status ec_mx_quantize_both(const void* x, int type, uint64_t batch, uint64_t rows,
                              uint64_t cols, uint64_t batch_stride, uint64_t stride,
                              void* row_codes, void* row_scales, void* col_codes,
                              void* col_scales, void* stream);

/* The same for rows grouped by offsets: the blocks of a column begin anew at
 * every group's first row, and group g's part of a column starts at the sum
 * of padded(rows) over the groups before it.  col_codes is
 * [cols][ec_mx_padded_groups(rows, groups) / 2]; elements past the last
 * group's part are not written.  Rows of no group are not written. */
ec_status ec_mx_quantize_groups(const void* x, int type, uint64_t rows, uint64_t cols,
                                uint64_t stride, const int32_t* offsets, uint32_t groups,
                                void* row_codes, void* row_scales, void* col_codes,
                                void* col_scales, void* stream);

/* y [rows][cols] (row stride `stride`) = the values of codes and scales,
 * rounded once to y's type. */
ec_status ec_mx_dequantize(const void* codes, const void* scales, uint64_t rows, uint64_t cols,
                           void* y, int type, uint64_t stride, void* stream);

/* y [rows][cols] = a b^T, summed in fp32 and rounded once: a [rows][depth]
 * and b [cols][depth] in the 4-bit form, depth a multiple of 128. */
ec_status ec_mx_product(const void* a_codes, const void* a_scales, uint64_t rows,
                        const void* b_codes, const void* b_scales, uint64_t cols, uint64_t depth,
                        void* y, int type, void* stream);

/* y [rows][cols]: row r of group e is a[r] b[e]^T with b [experts][cols][depth]. */
ec_status ec_mx_product_experts(const void* a_codes, const void* a_scales, uint64_t rows,
                                const void* b_codes, const void* b_scales, uint64_t cols,
                                uint64_t depth, const int32_t* offsets, uint32_t experts, void* y,
                                int type, void* stream);

/* y [experts][rows][cols]: y[e] = a[:, part e] b[:, part e]^T with a and b as
 * ec_mx_quantize_groups writes columns: [rows or cols][
 * ec_mx_padded_groups(tokens, experts)].  An expert without tokens gets 0. */
ec_status ec_mx_product_tokens(const void* a_codes, const void* a_scales, uint64_t rows,
                               const void* b_codes, const void* b_scales, uint64_t cols,
                               uint64_t tokens, const int32_t* offsets, uint32_t experts, void* y,
                               int type, void* stream);

/* What a product of these sizes runs as. ec_mx_product_tile: rows and columns
 * of a tile (256, 128 or 64; 16 where the kernel for few rows runs) in
 * ec_mx_product (experts = 0), ec_mx_product_experts, or, with tokens > 0,
 * ec_mx_product_tokens, where depth is not used; 0 if there is no such
 * product. ec_mx_product_rows_first: the rows that ec_mx_product puts into a
 * launch of their own, before one for the rest (0: all go in one). */
uint32_t ec_mx_product_tile(uint64_t rows, uint64_t cols, uint64_t depth, int type,
                            uint32_t experts, uint64_t tokens);
uint64_t ec_mx_product_rows_first(uint64_t rows, uint64_t cols, uint64_t depth, int type);

/* y [rows][cols] = Q(x) w^T: x [rows][depth] is quantized along its rows on
 * the way, w [cols][padded(depth)] is in the 4-bit form.  With experts > 0,
 * rows are grouped by offsets and w is [experts][cols][padded(depth)]; else
 * offsets is NULL.  The workspace (16-byte aligned, may be NULL where the
 * size is 0) holds ec_mx_linear_workspace_bytes(...) bytes. */
size_t ec_mx_linear_workspace_bytes(uint64_t rows, uint64_t depth, uint64_t cols,
                                    uint32_t experts);
ec_status ec_mx_linear(const void* x, int type, uint64_t rows, uint64_t depth, uint64_t stride,
                       const void* w_codes, const void* w_scales, uint64_t cols,
                       const int32_t* offsets, uint32_t experts, void* y, void* workspace,
                       size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EC_MX_H */
