/*
 * shampoo_experts.h - C ABI of the experts' path of a feed-forward block, next
 * to shampoo_layer.h: tokens sorted by expert and back, with weights applied,
 * and their gradients, for AMD Instinct MI355X (gfx950).
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

#ifdef __cplusplus
}
#endif
#endif /* SHAMPOO_EXPERTS_MI355X_H */
