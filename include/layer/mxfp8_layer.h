/*
 * mxfp8_layer.h -- C ABI of the training-layer operators of libmxfp8partial.so: what a layer
 * does with the MXFP8 weights that mxfp8_partial.h writes, on AMD Instinct MI355X (gfx950).
 *
 *  - mxfp8_matmul: the product of two 8-bit matrices with a scale for each block of 128 (or
 *    of 32, as the writeback's weights have): a layer's forward product, the gradient of its
 *    input, the gradient of its weight, for one token or many.
 *  - mxfp8_act_forward / mxfp8_act_backward: an activation function whose result leaves in 8
 *    bits for the next products and whose input is kept as a checkpoint in 8 bits; the
 *    backward pass reads that checkpoint.
 *  - mxfp8_layernorm_forward / mxfp8_layernorm_backward: layer norm, with the gradients of
 *    its weight and bias reduced over the rows.
 *
 * Conventions (those of mxfp8_partial.h, whose status codes, dtypes, mxfp8_buf and
 * mxfp8_last_error this header shares)
 *  - All buffer pointers are DEVICE pointers; the caller owns every buffer, workspaces
 *    included; the library allocates nothing, keeps no pointer after a call returns, never
 *    synchronizes, and enqueues its work on `hip_stream` (NULL = the null stream).
 *  - Calls that share a workspace must be ordered (one stream, or synchronized streams).
 *  - Matrices are row-major with a leading dimension in elements that is at least the row's
 *    width.  Element pointers need only their element's alignment.
 *  - 8-bit matrices hold E4M3 codes (OFP8 E4M3FN).  A block's values share one E8M0 scale
 *    byte s and stand for code * 2^(s - 127).  A row-wise block is 1 x 128 along a row, a
 *    column-wise block 128 x 1 down a column; the last block of a row or column may be
 *    shorter.  Row-wise scales are [rows][ld >= ceil(cols/128)], column-wise scales
 *    [ceil(rows/128)][ld >= cols].
 *  - The 8-bit outputs follow the rule of mxfp8_compute_scales and mxfp8_partial_cast:
 *    s = clamp(floor(log2 amax) - 8 + 127, 0, 254), 0 for amax 0; code = E4M3(x * 2^(127-s)),
 *    nearest even, saturated to +-448, the sign of zero kept.  amax is taken over the
 *    block's finite values; an infinity or NaN becomes the NaN code 0xFF, so it shows up in
 *    every product that reads it and costs its neighbours nothing.
 *  - Scale bytes that a call reads are at most 254 (not checked: device data).
 *  - Every check runs on the host before anything is enqueued; a call returns a status code
 *    and never aborts or throws.  A buffer that a call writes must not overlap any other
 *    buffer of the call (MXFP8_ERR_LAYOUT) except where stated.
 *  - Results do not depend on the order in which workgroups run: the same call on the same
 *    data gives the same bits.
 */
#ifndef MXFP8_LAYER_H
#define MXFP8_LAYER_H

#include "../mxfp8_partial.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ matrix product */

/* Where the direction that a product sums over lies in the stored array. */
typedef enum {
  MXFP8_ALONG_COLS = 0, /* array [outer][k]: the sum runs along each row   */
  MXFP8_ALONG_ROWS = 1  /* array [k][outer]: the sum runs down each column */
} mxfp8_along;

/* One 8-bit operand: outer x k values (outer = m for a, n for b).  A scale covers `block`
 * values along the sum and `across` outer values.  The weights of mxfp8_partial.h are
 * block 32, across 1: data_row / scale_row with ALONG_COLS, data_col / scale_col with
 * ALONG_ROWS.  The scale array is [ceil(outer/across)][scale_ld >= ceil(k/block)] with
 * ALONG_COLS and [ceil(k/block)][scale_ld >= ceil(outer/across)] with ALONG_ROWS. */
typedef struct {
  const void* data;  /* uint8 E4M3                                    */
  int64_t ld;        /* >= k (ALONG_COLS) or >= outer (ALONG_ROWS)    */
  const void* scale; /* uint8 E8M0                                    */
  int64_t scale_ld;
  int32_t along;     /* mxfp8_along                                   */
  int32_t block;     /* 32 or 128                                     */
  int32_t across;    /* 1 or 128                                      */
  int32_t reserved;  /* 0                                             */
} mxfp8_operand;

/* out[i][j] = round(sum over t < k of a(i, t) * b(j, t) + addend[i][j]), i < m, j < n. */
typedef struct {
  int64_t m, n, k;
  mxfp8_operand a, b;
  mxfp8_buf out;    /* out_dtype [m][ld >= n]                                            */
  mxfp8_buf addend; /* FP32 [m][ld >= n], or NULL; may be exactly `out` (same pointer and
                       ld, FP32), which adds the product to what is there                */
  int32_t out_dtype; /* MXFP8_FP32 or MXFP8_BF16                                         */
  int32_t reserved;  /* 0                                                                */
  void* workspace;   /* mxfp8_matmul_workspace() bytes, 16-byte aligned; may be NULL if 0 */
  int64_t workspace_bytes;
} mxfp8_product;

/* m == 0 or n == 0 is a valid no-op; k == 0 gives the addend, or zero.  With an FP32 output
 * every product is exact and sums are held in FP32 throughout.  With a BF16 output sums are
 * held in FP32, but the matrix unit aligns the products of each 8 successive values of the sum
 * to the largest of them and drops what lies below 2^-13 of it (as measured).  An element's
 * error beside the rounding to BF16 is so at most 2^-10 of its sum of |a b|.  On random data it
 * is 1.4e-5 of the result's norm, 1/100 of that rounding; where a sum cancels it may exceed the
 * rounding, and an FP32 output is the one to take.  Operand values count within FP32's normal
 * range: a smaller one may count as zero, a larger one as infinity. */
int mxfp8_matmul(const mxfp8_product* p, void* hip_stream);

/* Bytes of workspace that mxfp8_matmul needs for this product (0 if none), from its sizes,
 * types, leading dimensions and alignment alone; negative: the status code, negated, that
 * the call would return (a missing or short workspace aside).  Host-only. */
int64_t mxfp8_matmul_workspace(const mxfp8_product* p);

/* ------------------------------------------------------- activation with 8-bit checkpoint */

typedef enum {
  MXFP8_ACT_NONE = 0,  /* f(u) = u: a plain cast to 8 bits (forward only)               */
  MXFP8_ACT_GELU = 1,  /* f(u) = u / (1 + exp(-2 z)), z = sqrt(2/pi) (u + 0.044715 u^3) */
  MXFP8_ACT_SWIGLU = 2 /* f(g, u) = g / (1 + exp(-g)) * u                               */
} mxfp8_act_func;

/* An 8-bit matrix with block scales; data == NULL means absent. */
typedef struct {
  void* data;  /* uint8 E4M3 [rows][ld >= cols] */
  int64_t ld;
  void* scale; /* uint8 E8M0 */
  int64_t scale_ld;
} mxfp8_mat8;

/* An activation over rows x cols values.  SWIGLU has two inputs (gate first), the others
 * one; entries past a function's inputs are ignored.  A sigmoid below 2^-125 counts as 0: a
 * SWIGLU of a gate below -87.3 is 0 whatever finite value the other input has, and so are its
 * gradients. */
typedef struct {
  int64_t rows, cols;
  int32_t func;       /* mxfp8_act_func                                                   */
  int32_t dtype;      /* of input, grad and out: MXFP8_FP32 or MXFP8_BF16                 */
  mxfp8_buf input[2]; /* forward: the function's inputs [rows][ld >= cols]                */
  mxfp8_buf grad;     /* backward: gradient of the result [rows][ld >= cols]              */
  mxfp8_mat8 saved[2]; /* the inputs in row-wise blocks: forward writes those present,
                          backward reads them (all required)                              */
  mxfp8_buf out[2];   /* forward: out[0] = the result; backward: gradients of the inputs.
                         dtype; NULL = not wanted                                         */
  mxfp8_mat8 row[2];  /* the same values in row-wise blocks; NULL data = not wanted       */
  mxfp8_mat8 col[2];  /* the same values in column-wise blocks; NULL data = not wanted    */
} mxfp8_act;

/* f of the inputs.  Writes whichever of out[0], row[0], col[0], saved[] are present (at least
 * one; NONE takes no saved).  The function is evaluated in FP32 on the inputs themselves and
 * each output is rounded once from that value. */
int mxfp8_act_forward(const mxfp8_act* a, void* hip_stream);

/* Gradients of the inputs: grad times f's derivatives at the saved 8-bit inputs, for GELU and
 * SWIGLU.  Writes whichever of out[], row[], col[] are present (at least one). */
int mxfp8_act_backward(const mxfp8_act* a, void* hip_stream);

/* ------------------------------------------------------------------ layer norm */

/* y = (x - mean) * rstd * gamma + beta over rows of `cols` values, mean and rstd =
 * 1 / sqrt(variance + eps) per row (biased variance). */
typedef struct {
  int64_t rows, cols;
  int32_t dtype;      /* of x, y, dy, dx: MXFP8_FP32 or MXFP8_BF16                        */
  float eps;          /* forward; finite, >= 0                                            */
  mxfp8_buf x;        /* [rows][ld >= cols]                                               */
  const float* gamma; /* [cols]; NULL = all ones                                          */
  const float* beta;  /* forward: [cols]; NULL = none                                     */
  mxfp8_buf y;        /* forward: output; may be exactly x                                */
  float* mean;        /* [rows]: forward writes (NULL = not wanted), backward reads       */
  float* rstd;        /* [rows]: forward writes (NULL = not wanted), backward reads       */
  mxfp8_buf dy;       /* backward: gradient of y                                          */
  mxfp8_buf dx;       /* backward: gradient of x; NULL = not wanted; may be exactly dy    */
  float* dgamma;      /* backward: [cols]; NULL = not wanted                              */
  float* dbeta;       /* backward: [cols]; NULL = not wanted                              */
  void* workspace;    /* backward: mxfp8_layernorm_workspace() bytes, 16-byte aligned     */
  int64_t workspace_bytes;
} mxfp8_layernorm;

/* rows == 0 is a valid no-op; cols >= 1. */
int mxfp8_layernorm_forward(const mxfp8_layernorm* p, void* hip_stream);

/* dx = rstd (gamma dy - mean(gamma dy) - xh mean(gamma dy xh)), xh = (x - mean) rstd;
 * dgamma = sum over rows of dy xh; dbeta = sum over rows of dy (overwritten; zero for
 * rows == 0).  At least one of dx, dgamma, dbeta is required. */
int mxfp8_layernorm_backward(const mxfp8_layernorm* p, void* hip_stream);

/* Bytes of workspace mxfp8_layernorm_backward needs (0 if none), from rows, cols, dtype and
 * which outputs are present; negative: the status code, negated.  Host-only. */
int64_t mxfp8_layernorm_workspace(const mxfp8_layernorm* p);

#ifdef __cplusplus
}
#endif

#endif /* MXFP8_LAYER_H */
