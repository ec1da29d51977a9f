/*
 * shampoo_experts.h - C ABI of the experts' path of a feed-forward block, next
 * to shampoo_layer.h: tokens sorted by expert and back, with weights applied,
 * and matrix products in 8-bit floating point, dense or one matrix an expert;
 * with their gradients, for AMD Instinct MI355X (gfx950).
 *
 * Conventions are shampoo_layer.h's: status codes, shampoo_last_error, device
 * memory owned by the caller, every call asynchronous on the given stream,
 * row-major matrices with a leading dimension in elements, workspaces as
 * scratch of 256-byte alignment, pointers aligned to their element size,
 * deterministic results, fp32 sums, one rounding when a result is stored. An
 * output must not overlap an input or another output.
 */
#ifndef SHAMPOO_EXPERTS_MI355X_H
#define SHAMPOO_EXPERTS_MI355X_H

#include "shampoo.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------- tokens by expert
 * Slot j of token t, number t * slots + j, goes to expert ids[t][j]; an id
 * outside 0 .. experts - 1 leaves the slot out. Slots are put in order of their
 * experts, those of one expert in order of their numbers, and those left out
 * behind all others, likewise in order:
 *   offsets[e]  first row of expert e, offsets[experts]: rows in all
 *   rows[t][j]  the slot's row r; ~r (negative) if it is left out
 *   source[r]   the row's slot number; its ~ for a slot that is left out */
typedef struct {
  int64_t tokens;         /* >= 0, tokens * slots <= 2^31 - 1024        */
  int32_t slots, experts; /* 1 .. 1024 each                             */
  int32_t id_bytes;       /* 4 or 8: int32 or int64 ids                 */
  const void* ids;        /* tokens x slots, rows ld_ids elements apart */
  int64_t ld_ids;
  int32_t *offsets, *rows, *source; /* experts + 1, tokens x slots, tokens * slots */
} shampoo_sort_t;

/* Host only. Bytes of workspace (sizes are read). */
int shampoo_sort_workspace_size(const shampoo_sort_t* a, size_t* bytes_out);
int shampoo_sort_tokens(const shampoo_sort_t* a, void* workspace, size_t workspace_bytes, void* hip_stream);

/* With r = rows[t][j] of slots that are not left out:
 *   dispatch          xs[r] = x[t];  rows of slots left out: 0
 *   combine           y[t] = sum over j of weights[t][j] * ys[r]
 *   combine_backward  dys[r] = weights[t][j] * dy[t], rows of slots left out: 0;
 *                     dweights[t][j] = <dy[t], ys[r]>, 0 for a slot left out
 * Sums go over j in order. combine with weights = NULL (1) is the gradient of
 * dispatch. What a row or weight of a slot left out holds is not read. A value
 * of `rows` outside a plan's (over tokens * slots) counts as left out, and no
 * row is written for it. */
typedef struct {
  int64_t tokens, width;  /* tokens >= 0, width in [0, 2^21]; tokens * slots <= 2^31 - 1024 */
  int32_t slots;          /* 1 .. 1024                                  */
  int32_t dtype;          /* shampoo_dtype_t of x, ys, y, xs            */
  const int32_t* rows;    /* tokens x slots, as shampoo_sort_tokens wrote it */
  const float* weights;   /* tokens x slots, or NULL                    */
  const void *x, *ys;     /* x: tokens x width (dispatch: x, combine_backward: dy);
                             ys: tokens * slots x width (combine, combine_backward) */
  int64_t ld_x, ld_ys;
  void *y, *xs;           /* y: tokens x width (combine); xs: tokens * slots x width
                             (dispatch: xs, combine_backward: dys)      */
  int64_t ld_y, ld_xs;
  float* dweights;        /* combine_backward: tokens x slots           */
} shampoo_route_t;

int shampoo_dispatch(const shampoo_route_t* a, void* hip_stream);
int shampoo_combine(const shampoo_route_t* a, void* hip_stream);
int shampoo_combine_backward(const shampoo_route_t* a, void* hip_stream);

/* ------------------------------------------------- products in 8 bits
 * Q(v) of 128 values: scale 2^e, e the smallest integer >= -126 with max |v| <=
 * 448 * 2^e, and each v / 2^e rounded to e4m3 (to nearest even). An infinite or
 * NaN v becomes NaN and takes no part in the maximum. Powers of two, which the
 * matrix cores take as they are, make the rounding of v the only one.
 *   W^ = Q(W) by blocks of 128 x 128 of an in x out matrix,
 *   y = Qr(x) W^,  dx = Qr(dy) W^^T,  dW = Qc(x)^T Qc(dy)
 * with Qr by 128 columns of a row, Qc by 128 rows of a column, counted from
 * column 0 and from an expert's first row. Sums are taken for bf16 results by the
 * 8-bit matrix instruction: in fp32, but of eight neighbouring products each is cut
 * 14 bits below the largest (1.5e-5 of their root sum of squares if they are of one
 * size); for fp32 results by the bf16 instruction, in fp32 throughout, where values
 * of Q below 2^-126 may count as 0 and one that rounds up to 2^128 is infinite. What
 * is not finite makes every result it enters NaN, and leaves the others as they are.
 *
 * experts > 1 or offsets given: x's rows are sorted as shampoo_sort_tokens sorts
 * them, rows offsets[e] .. offsets[e + 1] (offsets[0] = 0, not falling, offsets[experts]
 * at most rows) meet matrix e; y and dx of rows behind the last expert's are 0,
 * and what x and dy hold there is not read. dW of an expert without rows is 0. */
typedef struct {
  int64_t in, out;    /* 1 .. 2^21                                        */
  int32_t experts;    /* matrices, 1 .. 1024                              */
  int32_t dtype;      /* shampoo_dtype_t of w                             */
  /* experts x in x out, rows ld_w, matrices stride_w elements apart: one behind the
     other (stride_w >= (in - 1) * ld_w + out) or side by side (stride_w >= out,
     (experts - 1) * stride_w + out <= ld_w). stride_w is read where experts > 1 */
  const void* w;
  int64_t ld_w, stride_w;
  /* Results. values: out rows of in values rounded up to a multiple of 128, 0
     behind in, 16-byte aligned; scales (exponent + 127, 1 byte) of the blocks:
     out / 128 rows of in / 128, both rounded up, rounded up to a multiple of 4,
     4-byte aligned. The backward ones, for dx (or NULL): the same with in and out
     exchanged. Matrices of experts follow each other. */
  void *values, *scales, *back_values, *back_scales;
} shampoo_weight8_t;

int shampoo_quantize_weight(const shampoo_weight8_t* a, void* hip_stream);

typedef struct {
  int64_t rows;           /* 0 .. 2^31 - 2^18: of y, dy, dx and of x; with saved
                             or dw at most 2^23 - 2^18                     */
  int64_t in, out;        /* 1 .. 2^21                                     */
  int32_t experts, dtype; /* matrices, 1 .. 1024; dtype of x, y, dy, dx, dw */
  const int32_t* offsets; /* experts + 1, or NULL: one matrix, all rows    */
  const int32_t* source;  /* NULL, or shampoo_sort_tokens' source: row r is row
                             source[r] / slots of x, which has x_rows      */
  int64_t x_rows;         /* >= 1 where rows >= 1; read with source        */
  int32_t slots;          /* 1 .. 1024; read with source                   */
  const int32_t* slot_rows; /* shampoo_sort_tokens' rows of the same plan, or NULL; read
                             with source, where rows is x_rows * slots     */
  /* as shampoo_quantize_weight wrote them (scales of 1 .. 254) */
  const void *values, *scales, *back_values, *back_scales;
  /* forward */
  const void* x;
  int64_t ld_x;
  void* y;
  int64_t ld_y;
  void* saved; /* shampoo_product8_saved_size bytes for dW: Qc(x); NULL: not kept */
  /* backward: reads saved, offsets and the backward values as in the forward
     pass; a NULL result is not computed */
  const void* dy;
  int64_t ld_dy;
  void* dx;
  int64_t ld_dx;
  void* dw; /* experts x in x out, apart as shampoo_weight8_t's w */
  int64_t ld_dw, stride_dw;
} shampoo_product8_t;

/* Host only. Bytes of `saved` (sizes are read). */
int shampoo_product8_saved_size(const shampoo_product8_t* a, size_t* bytes_out);
/* Host only. Bytes of workspace of shampoo_product8_forward (backward = 0) or
 * shampoo_product8_backward (1): sizes, and which pointers are NULL, are read. */
int shampoo_product8_workspace_size(const shampoo_product8_t* a, int32_t backward, size_t* bytes_out);
int shampoo_product8_forward(const shampoo_product8_t* a, void* workspace, size_t workspace_bytes, void* hip_stream);
int shampoo_product8_backward(const shampoo_product8_t* a, void* workspace, size_t workspace_bytes, void* hip_stream);

#ifdef __cplusplus
}
#endif
#endif /* SHAMPOO_EXPERTS_MI355X_H */
