/*
 * moe_fp4 -- 4-bit block-scaled matrices, their product, and the routing of
 * tokens to experts, for GB300 (sm_103a).  Companion of gemm_tn_f16.h, in the
 * same library and with the same conventions: plain C, device pointers on the
 * current device, asynchronous on `stream`, a gemm_status_t value returned,
 * arguments checked on the host before anything is launched, no device memory
 * allocated, every buffer owned by the caller.  What a call writes overlaps
 * nothing else of it: no matrix, no weights, none of the routing's arrays.
 *
 * Formats.  Rows are cut into blocks of neighbouring elements that share a
 * scale.  An element is E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives.
 *   FP4_NV  blocks of 16; scale E4M3, s = amax / 6 / 2^exponent rounded to
 *           nearest even (at most 448), one `exponent` for the whole matrix;
 *   FP4_MX  blocks of 32; scale E8M0, s = 2^(floor(log2 amax) - 2), exponent 0.
 * An element is x / (s 2^exponent) rounded to the nearest, ties to even, at
 * most 6 in magnitude; it stands for element * s * 2^exponent.  A block with a
 * NaN or an infinity in it (after the exponent is taken out) gets the NaN
 * scale, so that what is computed from it is NaN.
 *
 * Storage.  `codes`: rows of round_up(cols, 32) / 2 bytes, two elements a
 * byte, the even one in the low half, zeros past `cols`.  `scales`: tiles of
 * 128 rows; a tile is a run of 512-byte chunks, each 128 rows by 4 blocks with
 * row r's four bytes at 16 * (r % 32) + 4 * (r / 32), and columns padded (with
 * zero scales) to 256 elements: 4 chunks (FP4_NV) or 2 (FP4_MX) per 256.  This
 * is the order in which the tensor cores take scales, so that a product moves
 * them by whole chunks.  Rows are in groups (the experts of a weight, or the
 * rows of one expert), and a group starts a tile of its own:
 *   uniform groups of g rows:   group i's first tile is i * ceil(g / 128);
 *   groups given by offsets:    group i's first tile is offsets[i] / 128 + i.
 */
#ifndef MOE_FP4_H
#define MOE_FP4_H

#include "gemm_tn_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MOE_F16 = 0, MOE_BF16 = 1 };   /* types of activations and gradients */
enum { FP4_NV = 0, FP4_MX = 1 };      /* formats */

enum {
  FP4_MAX_COLS = 1 << 23,  /* columns of a 4-bit matrix */
  MOE_MAX_EXPERTS = 1024,  /* experts (groups) of a routing */
  MOE_MAX_TOP_K = 64,      /* slots per token */
  MOE_MAX_SLOTS = 1 << 30, /* tokens * top_k */
  MOE_MAX_HIDDEN = 1 << 30 /* elements of a row that is moved */
};

/* Where the slots of each token went: what moe_sort writes, as later calls
 * take it.  A slot p = token * top_k + j is one (token, expert) pair.  A program
 * that fills the arrays itself keeps to what moe_sort writes: `rows` a
 * permutation of 0 .. tokens * top_k - 1, `offsets` non-decreasing from 0 to at
 * most tokens * top_k, the rows from the last offset on those of dropped slots.
 * They are read on the device and not checked. */
typedef struct {
  int64_t tokens;
  int32_t top_k, experts;
  const int32_t* offsets;  /* experts + 1: expert e has rows offsets[e] .. offsets[e+1] - 1 */
  const int32_t* rows;     /* tokens * top_k: the row of each slot */
  const int32_t* ids;      /* tokens * top_k: the expert of each slot, as given to moe_sort.  No call
                              reads them after it: what they hold by then does not matter */
} moe_routing_t;

/* A 4-bit matrix. */
typedef struct {
  void* codes;             /* 16-byte aligned */
  void* scales;            /* 16-byte aligned, fp4_scale_bytes() of them */
  int64_t rows, cols;
  int32_t format;          /* FP4_* */
  int32_t exponent;        /* FP4_NV: -100 .. 100; FP4_MX: 0 */
  int32_t groups;          /* number of groups, at least 1 */
  int32_t reserved;        /* 0 */
  int64_t group_rows;      /* rows of a uniform group (groups * group_rows == rows) */
  const int32_t* offsets;  /* device, groups + 1, non-decreasing from 0 and at most `rows`;
                              NULL: uniform groups.  Rows past the last are in no group. */
} fp4_matrix_t;

/* Bytes of `codes` and `scales` for a matrix of these sizes; by_offsets: 1
 * when its groups are given by offsets.  No device is needed. */
int fp4_code_bytes(int64_t rows, int64_t cols, uint64_t* bytes);
int fp4_scale_bytes(int64_t rows, int64_t cols, int format, int groups, int by_offsets,
                    uint64_t* bytes);

/*
 * fp4_quantize: x (rows x cols of MOE_F16 or MOE_BF16, row stride ldx elements,
 * any 2-byte alignment) into `out`.
 *   routing == NULL: out->rows rows, in uniform groups (out->offsets NULL).
 *   routing != NULL: x has routing->tokens rows, and each is written to the rows
 *     of its slots: out->rows = tokens * top_k, out->groups = experts,
 *     out->offsets = routing->offsets.  Rows of dropped slots are not written.
 * Writes every scale of the matrix's groups, those of padding as zero when
 * uniform; codes past `cols` are zero.
 */
int fp4_quantize(const fp4_matrix_t* out, const void* x, int64_t ldx, int type,
                 const moe_routing_t* routing, void* stream);

/* fp4_dequantize: y (rows x cols of `type`, contiguous) = the values of `in`,
 * rounded to `type` (exact but for over- and underflow in MOE_F16); rows in no
 * group are zero. */
int fp4_dequantize(void* y, int type, const fp4_matrix_t* in, void* stream);

/*
 * fp4_gemm_tn: D[r][n] = alpha * sum_k a[r][k] * b[g(r)][n][k], fp32
 * accumulation, one rounding to `type`.
 *   a  rows of activations, in groups by offsets, or uniform;
 *   b  weights: as many uniform groups as a has, of group_rows = N rows each;
 *      same format and cols as a;
 *   D  a->rows x N of `type`, contiguous, 2-byte aligned, overlapping neither.
 * Rows of `a` in no group give zeros.  cols == 0 gives zeros.  alpha *
 * 2^(a's exponent + b's) has to be finite in fp32; it is rounded to fp32's 24 bits,
 * below its normal numbers too.
 * A pipeline wait that ran out (2 s) is reported by fp4_get_device_error().
 */
int fp4_gemm_tn(void* D, int type, const fp4_matrix_t* a, const fp4_matrix_t* b, float alpha,
                void* stream);

/* The same with a limit of its own for the kernel's waits (timeout_ns, 0: 2 s),
 * and inject = 1 for tests: the first stage of every CTA is never loaded, so that
 * a wait runs out, the call's result is undefined and the error word is set. */
int fp4_gemm_tn_ex(void* D, int type, const fp4_matrix_t* a, const fp4_matrix_t* b, float alpha,
                   uint64_t timeout_ns, int inject, void* stream);

/* The form that fp4_gemm_tn takes for `rows` rows in `groups` groups (uniform, or by
 * offsets) with n outputs each.  Host only, no GPU work; needs a current device
 * only to read its SM and cluster counts (with none, a GB300's are assumed). */
typedef struct {
  int cta_pair;            /* 1: tiles on CTA pairs */
  int split_k;             /* CTAs that share a tile's k; 1: none do */
  int tile;                /* outputs, and rows at most, of a tile */
  int box_rows;            /* rows of activations that one copy loads */
  int ctas;                /* launched */
} fp4_config_t;
int fp4_query_config(int64_t rows, int64_t n, int64_t cols, int format, int groups, int by_offsets,
                     fp4_config_t* out);

/* Waits for `stream`, a stream of the current device, then reads and clears its
 * error word of fp4_gemm_tn on that device: GEMM_OK or GEMM_ERR_TIMEOUT; `raw`
 * (may be NULL) gets code | site << 8.  Streams have a word each up to 63 of
 * them, beyond that they share. */
int fp4_get_device_error(void* stream, uint32_t* raw);

/*
 * moe_sort: slots sorted by expert.  ids: tokens * top_k expert numbers; any
 * outside [0, experts) marks a dropped slot.  rows[p] is slot p's place among
 * all slots ordered by expert, then by p, the dropped ones last; offsets[e] is
 * the first row of expert e and offsets[experts] the number of slots kept.
 * No two of the arrays overlap.
 */
int moe_sort(int32_t* offsets, int32_t* rows, const int32_t* ids, int64_t tokens, int top_k,
             int experts, void* stream);

/* moe_pairs: the inverse of rows: pairs[rows[p]] = p, for a program that walks
 * rows (none of the calls below needs it). */
int moe_pairs(int32_t* pairs, const moe_routing_t* routing, void* stream);

/* In what follows x, out and their gradients are tokens x hidden, y and its
 * gradient (tokens * top_k) x hidden in row order; all of `type` (2-byte
 * aligned), row strides equal to hidden but for ldx.  weights and their
 * gradient are tokens * top_k fp32 in slot order.  Sums are in fp32 in slot
 * order, rounded once. */

/* y[rows[p]] = x[p / top_k]; zeros in the rows of dropped slots. */
int moe_dispatch(void* y, const void* x, int64_t ldx, int64_t hidden, int type,
                 const moe_routing_t* routing, void* stream);

/* grad_x[t] = the sum over t's kept slots of grad_y[rows[p]]. */
int moe_dispatch_backward(void* grad_x, const void* grad_y, int64_t hidden, int type,
                          const moe_routing_t* routing, void* stream);

/* out[t] = the sum over t's kept slots of weights[p] * y[rows[p]].  Neither the
 * weight nor the row of a dropped slot is used, whatever they hold. */
int moe_combine(void* out, const void* y, const float* weights, int64_t hidden, int type,
                const moe_routing_t* routing, void* stream);

/* grad_y[rows[p]] = weights[p] * grad_out[p / top_k] and grad_weights[p] =
 * <grad_out[p / top_k], y[rows[p]]>; both zero for dropped slots.  Either of
 * grad_y and grad_weights may be NULL. */
int moe_combine_backward(void* grad_y, float* grad_weights, const void* grad_out, const void* y,
                         const float* weights, int64_t hidden, int type,
                         const moe_routing_t* routing, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FP4_H */
