/*
 * shampoo_layer.h - C ABI of the layer operators next to the Shampoo step:
 * the feed-forward half of a decoder layer, forward and backward, for AMD
 * Instinct MI355X (gfx950). Its weights are the [in][out] matrices that
 * shampoo_init registers, and the weight gradients it writes are what
 * shampoo_step reads.
 *
 * Conventions are shampoo.h's: status codes, shampoo_last_error, device
 * memory owned by the caller, every call asynchronous on the given stream,
 * row-major matrices with a leading dimension in elements. In addition:
 *  - Results are deterministic: every sum is taken in a fixed order.
 *  - Sums, statistics and products accumulate in fp32; an element is rounded
 *    (to nearest even) when it is stored in bf16.
 *  - A workspace is scratch: nothing is kept in it after the call's work on
 *    the stream. It must not be shared by calls that may run at once.
 *  - Pointers are aligned to their element size; workspace and saved to 256
 *    bytes. The block's products read 16-byte aligned bf16 matrices with ld a
 *    multiple of 8 (and, where a row is a product's summation index, cols a
 *    multiple of 8) in place; others, and fp32 ones as their three terms, are
 *    first copied to the workspace. Norms and dropout read any in place.
 *  - An output must not overlap an input or another output, except where
 *    said.
 */
#ifndef SHAMPOO_LAYER_MI355X_H
#define SHAMPOO_LAYER_MI355X_H

#include "shampoo.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------- gated feed-forward block
 *     g = x Wg,  u = x Wu,  h = act(g) * u,  y = h Wd
 * and, from dy,
 *     dh = dy Wd^T,  dg = dh * u * act'(g),  du = dh * act(g),
 *     dx = dg Wg^T + du Wu^T,
 *     dWg = x^T dg,  dWu = x^T du,  dWd = h^T dy.
 * x, y, dy, dx: tokens x d_model; Wg, Wu: d_model x d_hidden; Wd: d_hidden x
 * d_model. All of one dtype. bf16 products run on the bf16 matrix cores; fp32
 * operands are split exactly into three bf16 terms (as SHAMPOO_GEMM_SPLIT_BF16),
 * six products of which accumulate in fp32: every product of two elements keeps
 * an fp32 product's accuracy, whatever the sizes of the other elements (elements
 * under 2^-100 to 2^-126 absolute). Up to 64 tokens the forward pass takes the fp32
 * matrix instruction instead. An infinite or NaN operand makes every result it
 * enters non-finite, and leaves the others as they are. In bf16, g, u, h, dg
 * and du are rounded when they are stored between the products (h from unrounded
 * g and u): the matrix cores take no more of h, dg and du, and g and u are what a
 * step keeps. dx, dWg and dWu then differ from fp32 intermediates' by 0.003 in
 * relative norm, where rounding the results alone gives 0.0017. Up to 32 tokens
 * (d_model and d_hidden over 1) y is rounded alone: there h goes on as two bf16
 * terms; `saved` has the first. */
typedef enum {
  SHAMPOO_ACT_SILU = 0, /* g / (1 + exp(-g))                               */
  SHAMPOO_ACT_GELU = 1, /* tanh form                                       */
  SHAMPOO_ACT_RELU = 2  /* max(g, 0), derivative 0 at 0                    */
} shampoo_activation_t;

typedef struct {
  int64_t tokens, d_model, d_hidden; /* 0 <= tokens <= 2^31 - 1024; the others
                                        in [1, 2^21]                      */
  int32_t dtype;                     /* shampoo_dtype_t                      */
  int32_t activation;                /* shampoo_activation_t                 */
  const void *x, *w_gate, *w_up, *w_down;
  int64_t ld_x, ld_gate, ld_up, ld_down; /* cols <= ld <= 2^21, as all lds   */
  /* forward */
  void* y;
  int64_t ld_y;
  void* saved; /* shampoo_ffn_saved_size bytes for the backward pass: g, u and
                  h (fp32: its three terms); NULL: not kept (inference)    */
  /* backward (reads saved as the forward pass wrote it, with the same sizes,
     dtype and activation); a NULL result is not computed, dw_gate and dw_up
     together */
  const void* dy;
  int64_t ld_dy;
  void *dx, *dw_gate, *dw_up, *dw_down;
  int64_t ld_dx, ld_dw_gate, ld_dw_up, ld_dw_down;
} shampoo_ffn_t;

/* Host only. Bytes of `saved` (sizes and dtype are read). */
int shampoo_ffn_saved_size(const shampoo_ffn_t* a, size_t* bytes_out);
/* Host only. Bytes of workspace of shampoo_ffn_forward (backward = 0) or
 * shampoo_ffn_backward (1) for exactly this call: the alignment of the
 * pointers and the lds decide what is copied. */
int shampoo_ffn_workspace_size(const shampoo_ffn_t* a, int32_t backward, size_t* bytes_out);
int shampoo_ffn_forward(const shampoo_ffn_t* a, void* workspace, size_t workspace_bytes, void* hip_stream);
int shampoo_ffn_backward(const shampoo_ffn_t* a, void* workspace, size_t workspace_bytes, void* hip_stream);

/* A block behind a norm, shampoo_ffn_forward_normed (declared with the norms):
 * shampoo_ffn_forward for x = n of a shampoo_norm_forward call `norm` with z =
 * NULL, whose x, stats, weight and bias are still there. ReLU's derivative jumps
 * at 0, and the rounding of bf16 n moves g over it in one element of 2000, which
 * would make dx and dWg 2 to 4% wrong in norm. So for bf16 and ReLU g and u are
 * taken from n as it was before its rounding: what that left is made again as a
 * second term of x, for every element whose rounding is still x's own (else it
 * is 0). Its products run as those of over 32 tokens, and those of g and u take
 * twice as long. For other activations, whose results this would change by less
 * than their own roundings do, and for fp32 it is shampoo_ffn_forward itself. */

/* -------------------------- norms before and after a block, with dropout
 *     p = norm_post(z),  r = residual_scale x + drop(gate * p),
 *     n = norm_next(r)
 * z: the block's output, x: the residual stream before it, r: after it, n: the
 * next block's input. With z = NULL only n = norm_next(x) is computed (the
 * norm before a first block); r is then not written.
 *   norm(v) = (v - mean) / sqrt(var + eps) * weight + bias   (layer)
 *           = v / sqrt(mean(v^2) + eps) * weight + bias      (RMS)
 *           = v                                              (none)
 * weight and bias may be NULL (1 and 0). gate: one row of `width` factors for
 * each rows_per_gate consecutive rows (rows_per_gate >= rows: one for all; 1:
 * one a row); NULL: 1. n is taken from r before r is rounded.
 *
 * Dropout needs no mask in memory: the element (row, col) is kept where the
 * half-word col % 8 (low half of word 0 first) of Philox4x32-10(counter =
 * (col / 8, row mod 2^32, row / 2^32, offset), key = (seed mod 2^32, seed /
 * 2^32)) is at least T = round(65536 p), and multiplied by 65536 / (65536 -
 * T); others become 0. It depends on nothing else: not on strides, dtype,
 * launch or direction. */
typedef enum { SHAMPOO_NORM_NONE = 0, SHAMPOO_NORM_RMS = 1, SHAMPOO_NORM_LAYER = 2 } shampoo_norm_kind_t;

typedef struct {
  int64_t rows, width; /* 0 <= rows <= 2^40, 1 <= width <= 8192        */
  int32_t dtype;       /* shampoo_dtype_t of every array but stats     */
  int32_t post_kind, next_kind;
  float eps;            /* > 0                                         */
  float residual_scale; /* finite                                      */
  double dropout;       /* p, 0 <= p < 1                               */
  uint64_t seed;
  uint32_t offset; /* another one for each call under one seed         */
  int64_t rows_per_gate;
  const void *z, *x;
  int64_t ld_z, ld_x;
  void *r, *n; /* n: NULL where next_kind is none. r may be x or z itself
                  (same pointer and ld) in the forward pass              */
  int64_t ld_r, ld_n;
  const void *post_weight, *post_bias, *gate, *next_weight, *next_bias;
  int64_t ld_gate;
  float* stats; /* rows x 4, 16-byte aligned: written by the forward pass
                   (NULL: not kept), read by the backward pass           */
  /* backward: reads z, r (x where z is NULL), gate, weights and stats */
  const void *dr, *dn; /* gradients of r and n; dr NULL: 0; dn NULL where
                          next_kind is none                              */
  int64_t ld_dr, ld_dn;
  void *dx, *dz; /* may be dr or dn themselves; NULL: not wanted         */
  int64_t ld_dx, ld_dz;
  void *d_post_weight, *d_post_bias, *d_gate, *d_next_weight, *d_next_bias;
  int64_t ld_d_gate;
} shampoo_norm_t;

/* Host only. Bytes of workspace of shampoo_norm_backward. */
int shampoo_norm_workspace_size(const shampoo_norm_t* a, size_t* bytes_out);
int shampoo_norm_forward(const shampoo_norm_t* a, void* hip_stream);
int shampoo_norm_backward(const shampoo_norm_t* a, void* workspace, size_t workspace_bytes, void* hip_stream);

/* The block behind the norm (above). Host only: its bytes of workspace. */
int shampoo_ffn_normed_workspace_size(const shampoo_ffn_t* a, const shampoo_norm_t* norm, size_t* bytes_out);
int shampoo_ffn_forward_normed(const shampoo_ffn_t* a, const shampoo_norm_t* norm, void* workspace, size_t workspace_bytes,
                               void* hip_stream);

/* ------------------------------------------------------------- dropout
 * y = x where kept (times the scale above), else 0; y may be x itself. Its
 * gradient is the same call on dy. */
typedef struct {
  int64_t rows, cols; /* 0 <= rows <= 2^40, 0 <= cols <= 2^31 - 1024 */
  int32_t dtype;
  uint32_t offset;
  double dropout;
  uint64_t seed;
  const void* x;
  void* y;
  int64_t ld_x, ld_y;
} shampoo_dropout_t;

int shampoo_dropout(const shampoo_dropout_t* a, void* hip_stream);

#ifdef __cplusplus
}
#endif
#endif /* SHAMPOO_LAYER_MI355X_H */
