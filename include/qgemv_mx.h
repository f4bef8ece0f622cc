/*
 * qgemv_mx.h -- prompts over MXFP4 weights on an AMD Instinct MI355X (gfx950):
 * quantisation to MXFP4, products for any number of tokens, products of tokens
 * sorted by expert, and the sort itself with the way back and its gradient.
 * Part of libqgemv.so; qgemv.h holds the formats, the status codes and the
 * conventions, which hold here too (host-side validation before any HIP call,
 * a refused call enqueues nothing and leaves every output untouched, caller's
 * memory and stream, no waiting, no allocation, re-entrant calls, safe under
 * stream capture), but for the products' order of sums (see qgemv_rows_mx).
 * The caller's current device must be the buffers' and the stream's device.
 *
 * A prompt through a mixture of experts whose weights stay in their GGUF
 * blocks (neurostream README, "How it works": the router names the experts,
 * each expert's rows are one window of the stacked tensor; gate and up are one
 * phase, down the next):
 *
 *     qgemv_expert_sort(ids)                     places of (token, choice) slots
 *     qgemv_expert_mx_swiglu(gate, up, x, slots) h, in the experts' order
 *     qgemv_expert_mx(down, h)                   y, in the experts' order
 *     qgemv_expert_combine(y, pos, w)            one weighted sum per token
 *
 * with qgemv_mx_quantize before a product where the activations are to be
 * 4-bit too.  Every id, count and place stays on the device.
 *
 * Outputs of one call do not depend on timing, the stream or earlier calls: no
 * kernel uses floating-point atomics.
 */
#ifndef QGEMV_MX_H
#define QGEMV_MX_H

#include "qgemv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of a qg_tensor besides the block format QG_MXFP4. */
enum qg_float { QG_F32 = 32, QG_F16 = 33, QG_BF16 = 34 };

/* Most experts of one stacked tensor. */
#define QG_MAX_EXPERTS 1024

/* Rows of activations in device memory.  Float types: row r starts at element
 * r * stride of data, elements contiguous, data aligned to one element; an
 * input may have any stride >= 0, an output's must be >= n_cols where it has
 * more than one row.  QG_MXFP4 (inputs of the products only): rows of
 * n_cols / 32 blocks, back to back, data 16-byte aligned, stride == n_cols;
 * as of weights, the whole 16-byte granule of the last byte may be read.
 * Inputs and outputs of one call must not overlap. */
typedef struct qg_tensor {
  void *data;
  int32_t type;     /* enum qg_float, or QG_MXFP4 */
  int32_t reserved; /* must be 0 */
  int64_t n_rows;   /* 0 .. 2^31 - 2^16 (QG_E_SHAPE above, as of a matrix' rows) */
  int64_t n_cols;   /* 0 .. 2^31 - 2^16 */
  int64_t stride;   /* elements between rows */
} qg_tensor;

/* Statuses of these calls beyond the meanings in qgemv.h: QG_E_FMT an element
 * type or weight format the call does not take; QG_E_SHAPE sizes that do not
 * fit each other or are out of range; QG_E_ARG strides, alignment, reserved
 * fields, counts. */

/* Quantises the rows of x (QG_F32, QG_F16 or QG_BF16) into q's MXFP4 blocks
 * (q->fmt QG_MXFP4, q->n_rows = x->n_rows, q->k = x->n_cols; q->data is
 * written, exactly q->n_bytes).  Per block of 32 values with a = max|x|:
 *     e = clamp(floor(log2 a) - 2 + 127, 0, 254)   (e = 0 where a = 0),
 *     code = x * 2^(127 - e) rounded to the nearest E2M1 value, ties to the
 *            even code, magnitudes above 6 to 6, signs kept (zeros' too);
 * the OCP MX v1.0 conversion, exact up to that one rounding.  A block that
 * holds an infinity or a NaN gets e = 255: all its values decode to NaN. */
int qgemv_mx_quantize(const qg_tensor *x, const qg_matrix *q, qg_stream_t stream);

/* The values of rows [row_start, row_end) of q, rounded once to out's type
 * (out->n_rows = row_end - row_start, out->n_cols = q->k): exact in QG_F32
 * and QG_BF16 (but for magnitudes of 2^128 and more, which are above their range
 * and give infinities: 2, 3, 4 and 6 at scale 254, 4 and 6 at 253), rounded in
 * QG_F16. */
int qgemv_mx_dequantize(const qg_matrix *q, int64_t row_start, int64_t row_end, const qg_tensor *out,
                        qg_stream_t stream);

/* y[t] = W[row_start:row_end] . x[t] for every row t of x, W in MXFP4: any
 * number of tokens on the matrix cores (neurostream README, "What the numbers
 * taught us": tokens that share one pass over the weights cost about one
 * token's weight traffic).  x->n_cols = w->k; y->n_rows = x->n_rows, y->n_cols
 * = row_end - row_start, y a float type.  x may be
 *   QG_F32, QG_F16, QG_BF16  taken exactly: a weight below 2^128 is exact in
 *             bf16, and x is the exact sum of three, two or one bf16 terms (but
 *             for bits of QG_F32 below 2^-133, where bf16's subnormals end: cut
 *             off).  Rows with weights of 2^128 and more (scales 253 and 254,
 *             which qgemv_mx_quantize never writes) are summed in 64 bits, and
 *             slowly;
 *   QG_MXFP4  4-bit activations (qgemv_mx_quantize), codes and scales of both
 *             sides multiplied by the scaled 4-bit matrix instructions.
 * Products are exact, sums are fp32 in the matrix cores' order, y is rounded
 * once (a sum past fp32's range is infinite).  An output is the same for any stream and run, and for windows of as
 * many rows wherever they begin; unlike the calls of qgemv.h, its order of sums
 * may differ for another number of tokens or of rows in the window, by which
 * the kernel is chosen.  Non-finite values follow IEEE
 * arithmetic of x times W, with the scale 255 as NaN.  No rows or no tokens
 * do nothing. */
int qgemv_rows_mx(const qg_matrix *w, int64_t row_start, int64_t row_end, const qg_tensor *x, const qg_tensor *y,
                  qg_stream_t stream);

/* h[t] = silu(gate[rows] . x[t]) * (up[rows] . x[t]), both products and the
 * SiLU in fp32 (qgemv_silu_mul's; below -87.3, where silu is less than 2^-119
 * in magnitude, it gives 0), rounded once.  gate and up match in n_rows
 * and k (else QG_E_SHAPE); otherwise as qgemv_rows_mx. */
int qgemv_rows_mx_swiglu(const qg_matrix *gate, const qg_matrix *up, int64_t row_start, int64_t row_end,
                         const qg_tensor *x, const qg_tensor *h, qg_stream_t stream);

/* Stable sort of n_tok * n_sel slots by expert.  ids: device, n_tok x n_sel,
 * slot i = t * n_sel + s holds the id of token t's choice s; an id outside
 * [0, n_expert) belongs to no expert (a padded token, a dropped choice).
 *   offsets (n_expert + 1): offsets[e] = slots of experts below e; the last is
 *            the number of kept slots
 *   slots   (n_tok * n_sel): the slot at each place, by expert and then by
 *            slot; -1 behind the last kept one
 *   pos     (n_tok * n_sel): each slot's place, -1 for a dropped one
 * All int32 device arrays.  n_tok * n_sel <= 2^30, n_sel >= 1,
 * 1 <= n_expert <= QG_MAX_EXPERTS.  n_tok = 0 writes the zero offsets. */
int qgemv_expert_sort(const int32_t *ids, int64_t n_tok, int32_t n_sel, int64_t n_expert, int32_t *offsets,
                      int32_t *slots, int32_t *pos, qg_stream_t stream);

/* The experts' products over sorted places: for expert e and places p in
 * [offsets[e], offsets[e + 1]),
 *     y[p] = W[e * out : (e + 1) * out] . x[src],  src = slots[p] / n_sel,
 * or src = p where slots is NULL (x already in the experts' order; n_sel is
 * then ignored).  w holds n_expert stacked matrices of out rows (QG_E_SHAPE
 * otherwise); y->n_rows is the number of places the arrays offer (at least
 * the last offset), y->n_cols = out; without slots x->n_rows >= y->n_rows.
 * Each weight is read once per tile of its expert's places; experts without a
 * token cost nothing.  Rows of y behind the last offset stay as they were.
 * Offsets are clamped to [0, y->n_rows]; a src outside x's rows gives a
 * row of zeros.  x, y and arithmetic as qgemv_rows_mx; the order of sums may
 * differ for another number of places, experts or rows of one, but does not
 * depend on how the places are shared out. */
int qgemv_expert_mx(const qg_matrix *w, int64_t n_expert, const qg_tensor *x, const int32_t *offsets,
                    const int32_t *slots, int32_t n_sel, const qg_tensor *y, qg_stream_t stream);

/* The same for the SwiGLU pair: h[p] = silu(gate_e . x[src]) * (up_e . x[src]). */
int qgemv_expert_mx_swiglu(const qg_matrix *gate, const qg_matrix *up, int64_t n_expert, const qg_tensor *x,
                           const int32_t *offsets, const int32_t *slots, int32_t n_sel, const qg_tensor *h,
                           qg_stream_t stream);

/* out[p] = x[slots[p] / n_sel] for p < out->n_rows: tokens in the experts'
 * order (the products above do this as they load).  Same float type and
 * n_cols; slots holds out->n_rows entries.  Rows whose slot is negative, or
 * names a token x does not have, stay as they were. */
int qgemv_expert_gather(const qg_tensor *x, const int32_t *slots, int32_t n_sel, const qg_tensor *out,
                        qg_stream_t stream);

/* The way back: out[t] = sum_s w[t, s] y[pos[t, s]] (neurostream README, "How
 * it works": the router's weights mix the experts' outputs), one fp32 fma per
 * term in s order, rounded once to out's type.  pos: device, out->n_rows x
 * n_sel; w: device, the same shape, or NULL for weights of 1, which is also
 * the gradient of qgemv_expert_gather (dx from dout).  Places that are
 * negative or beyond y's rows add nothing; a token without any gets zeros.
 * 0 <= n_sel <= 2^30. */
int qgemv_expert_combine(const qg_tensor *y, const int32_t *pos, const float *w, int32_t n_sel,
                         const qg_tensor *out, qg_stream_t stream);

/* The gradient of qgemv_expert_combine from dout (n_tok rows):
 *     dy[pos[t, s]] = w[t, s] dout[t],   dw[t, s] = <dout[t], y[pos[t, s]]>,
 * both products in fp32, dw's sum in a fixed order, 0 where pos is dropped.
 * dy has y's type and rows; rows no pos names stay as they were.  A place is
 * named at most once, as the sort's are.  y and dy may not be the same
 * memory.  n_sel >= 1; w is required. */
int qgemv_expert_combine_grad(const qg_tensor *dout, const qg_tensor *y, const int32_t *pos, const float *w,
                              int32_t n_sel, const qg_tensor *dy, float *dw, qg_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QGEMV_MX_H */
