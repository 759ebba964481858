/*
 * linear -- linear layers in 16 bits with what stands around their product:
 * bias, activation and residual, dense or with each row's expert's weights,
 * and their gradients, for GB300 (sm_103a).  Companion of gemm_tn_f16.h and
 * moe_fp4.h, in the same library and with the same conventions: plain C, device
 * pointers on the current device, asynchronous on `stream`, a gemm_status_t
 * value returned, arguments checked on the host before anything is launched, no
 * device memory allocated, every buffer owned by the caller.  What a call writes
 * overlaps nothing else of it.
 *
 * For a row r of x and its group g (the whole matrix, or the expert it belongs to)
 *
 *   z[r][n]   = sum_h x[r][h] w[g][n][h] + bias[g][n]
 *   out[r][n] = act(z[r][n]) + residual[r][n]
 *
 * and with dz[r][n] = grad_out[r][n] act'(z[r][n])
 *
 *   grad_x[r][h]     = sum_n dz[r][n] w[g][n][h]
 *   grad_w[g][n][h]  = sum over the rows r of g of dz[r][n] x[r][h]
 *   grad_bias[g][n]  = sum over the rows r of g of dz[r][n]
 *
 * (the residual's gradient is grad_out).  Everything is of one type, MOE_F16 or
 * MOE_BF16.  Sums are in fp32; z, out and the gradients are rounded once.  dz is
 * rounded to the type before the products with it, which take 16-bit operands;
 * grad_bias is the sum of dz before that.
 *
 * Activations: LINEAR_NONE z; LINEAR_RELU max(z, 0), with slope 0 at 0;
 * LINEAR_GELU z P(Z <= z) for a standard normal Z; LINEAR_GELU_TANH
 * z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2; LINEAR_SILU z / (1 + e^-z).
 */
#ifndef LINEAR_H
#define LINEAR_H

#include "moe_fp4.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { LINEAR_NONE = 0, LINEAR_RELU = 1, LINEAR_GELU = 2, LINEAR_GELU_TANH = 3, LINEAR_SILU = 4 };

enum {
  LINEAR_MAX_COLS = 1 << 23, /* inputs, and outputs, of a layer */
  LINEAR_MAX_ROWS = 1 << 30  /* rows */
};

/* The layer.  Matrices are row by row, 2-byte aligned at least, with rows that do
 * not overlap: a row stride (elements) is at least the width, and the arrays
 * without one are contiguous.  Rows that start on 16-byte boundaries (pointer
 * and stride) are read where they are, and so are all rows of forward products of few
 * rows; others are first copied to `workspace`. */
typedef struct {
  int64_t rows;              /* of x and out */
  int64_t in, out;           /* elements of their rows */
  int32_t type;              /* MOE_F16 or MOE_BF16 */
  int32_t activation;        /* LINEAR_* */
  const void* x;             /* rows x in */
  int64_t ldx;
  const void* w;             /* experts x out x in, an expert's rows `ldw` apart */
  int64_t ldw;
  /* NULL: one group, all rows.  Otherwise rows are in expert order, rows ==
   * tokens * top_k, and expert e has its own out x in weights (and `out` biases),
   * one expert's after the other's: expert e's begin at row e * out.  Of the
   * routing the offsets are read alone.  Rows past the last offset are in no
   * expert: they give zeros, and their values affect nothing. */
  const moe_routing_t* routing;
} linear_t;

/* For tests and measurements; NULL, or all zero, chooses.  `tile` not 0: the call's
 * products take the form of these three (see linear_config_t; one that there is
 * not is GEMM_ERR_INVALID_VALUE).  timeout_ns: the limit of a wait in the kernels,
 * 0: 2 s, and 1 us for each 64 elements of a product's sums.  inject = 1: the first
 * stage of every CTA is never loaded, so that a wait runs out, the results are
 * undefined and the error word is set. */
typedef struct {
  int cta_pair, tile, split_k;
  int inject;
  uint64_t timeout_ns;
} linear_options_t;

/* linear_forward: out (rows x out, contiguous) and, where `preact` is not NULL, z
 * (the same, rounded).  bias (experts x out) and residual (rows x out, row stride
 * ldr; dense layers alone) may be NULL.  in == 0: the sums are zero. */
int linear_forward(void* out, void* preact, const linear_t* layer, const void* bias,
                   const void* residual, int64_t ldr, void* workspace, uint64_t workspace_bytes,
                   const linear_options_t* opt, void* stream);

/* linear_backward: those of grad_x (rows x in), grad_w (experts x out x in) and grad_bias
 * (experts x out) that are not NULL, all contiguous.  grad_out: rows x out, row stride
 * ldg.  preact: rows x out, contiguous, as linear_forward wrote it; NULL for
 * LINEAR_NONE.  layer->x is read for grad_w alone and layer->w for grad_x alone,
 * and may be NULL otherwise.  The gradients of an expert without rows are zero.  The bits of a
 * gradient do not depend on which others the call is for. */
int linear_backward(void* grad_x, void* grad_w, void* grad_bias, const linear_t* layer,
                    const void* grad_out, int64_t ldg, const void* preact, void* workspace,
                    uint64_t workspace_bytes, const linear_options_t* opt, void* stream);

/* Bytes of workspace that the call with these pointers needs (they are not
 * dereferenced; their alignment counts).  It is 16-byte aligned, its contents do
 * not matter before or after, and calls that may run at once need one each.
 * Host only. */
int linear_forward_workspace(const linear_t* layer, const linear_options_t* opt, uint64_t* bytes);
int linear_backward_workspace(const void* grad_x, const void* grad_w, const void* grad_bias,
                              const linear_t* layer, const void* grad_out, int64_t ldg,
                              uint64_t* bytes);

/* The products of these calls.  grad_x and grad_w of one call share the GPU, and may be cut in
 * another way than either in a call without the other one: _OF_BOTH is the former. */
enum {
  LINEAR_FORWARD = 0,
  LINEAR_GRAD_X = 1,
  LINEAR_GRAD_W = 2,
  LINEAR_GRAD_X_OF_BOTH = 3,
  LINEAR_GRAD_W_OF_BOTH = 4
};

/* How a product is cut. */
typedef struct {
  int cta_pair;              /* 1: 256 x 256 tiles on CTA pairs; 0: 128 x tile on single CTAs */
  int tile;                  /* rows of a tile (grad_w: outputs): 256; on single CTAs also 64, 128
                                and, but for grad_w, 32; forward without the tensor cores: 1, 2,
                                4, 8 rows at a time */
  int split_k;               /* CTAs of a cluster (there: warps) that share a tile's sums, 1, 2, 4
                                or 8; 1: none do */
  int ctas;                  /* launched */
} linear_config_t;

/* The form that a product of a layer of these sizes takes (experts: 0 for a dense
 * one).  Host only, no GPU work; needs a current device only to read its SM
 * and cluster counts (with none, a GB300's are assumed). */
int linear_query_config(int product, int64_t rows, int64_t in, int64_t out, int experts,
                        linear_config_t* config);

/* Waits for `stream`, a stream of the current device, then reads and clears its
 * error word of these calls on that device: GEMM_OK or GEMM_ERR_TIMEOUT; `raw`
 * (may be NULL) gets code | site << 8.  Streams have a word each up to 63 of
 * them, beyond that they share. */
int linear_get_device_error(void* stream, uint32_t* raw);

#ifdef __cplusplus
}
#endif

#endif /* LINEAR_H */
