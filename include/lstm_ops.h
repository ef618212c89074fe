/*
 * lstm_ops.h -- operators that stand beside the recurrent layers of lstm.h in
 * a sequence model: linear attention with a decay for each head (a recurrent
 * layer whose state is a matrix, parallel over time for prompts and
 * training), layer norm, and the AdamW step over many tensors.
 *
 * Conventions are those of lstm.h: device memory of the current device, owned
 * by the caller; scratch in a caller's workspace whose size a query gives; a
 * stream argument (NULL = default stream); an lstm_status from every call;
 * host checks before anything is enqueued; no exception crosses the
 * interface; nothing is allocated.  Calls may be captured into a graph.
 * Dtypes: LSTM_F32 and LSTM_BF16.  Sums, states and statistics are fp32, and
 * so is all arithmetic but for two operands of whole bf16 sequences (see
 * lstm_linear_attention_forward).
 */
#ifndef LSTM_AMD_LSTM_OPS_H
#define LSTM_AMD_LSTM_OPS_H

#include <stddef.h>

#include "lstm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------- linear attention
 * Per batch row and head h, with a state S [key_dim, value_dim] and
 * gamma_h = exp(log_decay[h]):
 *     S_t = gamma_h S_{t-1} + k_t v_t^T        o_t = scale * q_t S_t
 * Query head h reads key/value head h / (heads / kv_heads). */

/* A [T, B, heads, dim] tensor of the call's dtype: element strides of the
 * time, batch and head axes; the last axis is dense.  Any strides and any
 * alignment are taken for an input (0 repeats it), the time stride below 2^31
 * bytes; an output must not overlap itself, which is the caller's to keep.
 * Addresses are 64-bit. */
typedef struct {
    void *data;
    long long time, batch, head;
} lstm_view;

typedef struct {
    int dtype;               /* lstm_dtype of q, k, v, o and their gradients */
    int T, B;                /* >= 1; T at most 2^31 - 2^15 - 1 */
    int heads, kv_heads;     /* >= 1, heads a multiple of kv_heads */
    int key_dim, value_dim;  /* 1..256 */
    float scale;             /* finite, not 0 */
} lstm_linear_attention_shape;

/* Bytes of workspace (0 is possible) of the forward and of the backward call
 * of this shape.  Touches no device. */
lstm_status lstm_linear_attention_workspace_size(const lstm_linear_attention_shape *shape, size_t *bytes);
lstm_status lstm_linear_attention_backward_workspace_size(const lstm_linear_attention_shape *shape, size_t *bytes);

/* Whole sequences.
 *   q, k, v      views with heads, kv_heads and kv_heads heads
 *   log_decay    [heads] float32, at most 0 (-infinity: gamma = 0, o_t reads
 *                token t alone); a positive one grows without a bound
 *   lengths      [B] int32 DEVICE memory, or NULL (every row has T tokens);
 *                values are clamped to 0..T.  Tokens past a row's length are
 *                not read, their o is 0, and the row's state passes them by.
 *   state        [B, heads, key_dim, value_dim] float32, the state before the
 *                first token, or NULL (zeros)
 *   o            view with heads heads, written
 *   state_out    like state: the state after each row's last token, or NULL.
 *                It may be the memory of `state` (then updated in place).
 * LSTM_BF16: o is rounded to bf16, and so are two operands of the matrix
 * instructions on the way to it: the state where a chunk's tokens read it, and
 * the decayed q k^T inside a chunk (o is off by 0.0023 of its size, rms; its
 * own rounding alone is 0.0017).  The state itself is summed in fp32, from
 * products to 2^-24 (to 2^-17 where it is not returned and so enters bf16
 * results only).  The gradients are computed alike.  A single token
 * (lstm_linear_attention_step) rounds o alone, so a prompt and its tokens one
 * by one differ by those operands' roundings.
 * LSTM_ERR_ARG: NULL argument, a dim outside 1..256, heads not a multiple of
 * kv_heads, a scale that is 0 or not finite; LSTM_ERR_SHAPE: T or B < 1, T
 * above its limit, B * heads above 2^20, a time stride of 2^31 bytes;
 * LSTM_ERR_WORKSPACE: workspace too short.  Sequences run in chunks of 32
 * tokens: a value that is not finite spoils its row's later outputs and may
 * spoil earlier ones of its chunk. */
lstm_status lstm_linear_attention_forward(const lstm_linear_attention_shape *shape, const lstm_view *q,
                                          const lstm_view *k, const lstm_view *v, const float *log_decay,
                                          const int *lengths, const float *state, const lstm_view *o,
                                          float *state_out, void *workspace, size_t workspace_bytes, void *stream);

/* Gradients of that forward.  do_: gradient of o; dstate_out: gradient of
 * state_out, or NULL (zeros); dq, dk, dv: views with the heads of q, k, v,
 * written; dstate: gradient of state, or NULL (not wanted).  The decay is a
 * constant of the layer and gets no gradient.  Tokens past a row's length get
 * zero gradients.  Outputs must not overlap inputs.  A key or value head shared by several query heads gets the
 * sum of their gradients, in head order. */
lstm_status lstm_linear_attention_backward(const lstm_linear_attention_shape *shape, const lstm_view *q,
                                           const lstm_view *k, const lstm_view *v, const float *log_decay,
                                           const int *lengths, const float *state, const lstm_view *do_,
                                           const float *dstate_out, const lstm_view *dq, const lstm_view *dk,
                                           const lstm_view *dv, float *dstate, void *workspace,
                                           size_t workspace_bytes, void *stream);

/* One token for each of B requests (shape->T must be 1; the views' time
 * strides are not used).  pool [n_slots, heads, key_dim, value_dim] float32
 * holds the requests' states and is updated in place.
 *   slots  [B] int32 device memory: row b's state is pool[slots[b]]; a value
 *          outside 0..n_slots-1 marks an idle row, whose o is 0.  Two rows of
 *          one call must not name the same slot.  NULL: row b uses slot b
 *          (n_slots >= B, else LSTM_ERR_SHAPE). */
lstm_status lstm_linear_attention_step(const lstm_linear_attention_shape *shape, const lstm_view *q,
                                       const lstm_view *k, const lstm_view *v, const float *log_decay,
                                       const int *slots, int n_slots, float *pool, const lstm_view *o, void *stream);

/* ----------------------------------------------------------------- layer norm
 * Over rows of `width` values: z = x + residual (rounded to the dtype),
 *     mean = sum z / width, rstd = 1 / sqrt(sum (z - mean)^2 / width + eps),
 *     y = (z - mean) rstd weight + bias.
 *   x, residual, y, sum  [rows, width] dtype, rows x_stride (residual_stride,
 *                ...) elements apart, at least width; y and sum are dense
 *   residual     or NULL (z = x; then sum must be NULL)
 *   weight, bias [width] dtype, or NULL (1 and 0)
 *   sum          receives z, or NULL
 *   mean, rstd   [rows] float32, or NULL
 * rows >= 0 (0 does nothing), width in 1..2^28, eps >= 0 and finite.  y may be x's
 * memory, and sum may be residual's or x's, where the rows are dense. */
lstm_status lstm_layer_norm_forward(int dtype, const void *x, long long x_stride, const void *residual,
                                    long long residual_stride, const void *weight, const void *bias,
                                    long long rows, int width, float eps, void *y, void *sum, float *mean,
                                    float *rstd, void *stream);

lstm_status lstm_layer_norm_backward_workspace_size(long long rows, int width, size_t *bytes);

/* Gradients.  z: the x of the forward, or its sum where it had a residual;
 * mean, rstd: as the forward wrote them; dsum [rows, width] dense: gradient
 * that reaches z from elsewhere (the residual stream), or NULL.
 *   dx        [rows, width] dtype, dense: gradient of z (of x, and of the
 *             residual); may be dsum's or dense dy's memory
 *   dweight, dbias  [width] dtype, or NULL; their sums over the rows run in a
 *             fixed order. */
lstm_status lstm_layer_norm_backward(int dtype, const void *dy, long long dy_stride, const void *z,
                                     long long z_stride, const float *mean, const float *rstd, const void *weight,
                                     const void *dsum, long long rows, int width, void *dx, void *dweight,
                                     void *dbias, void *workspace, size_t workspace_bytes, void *stream);

/* --------------------------------------------------------------------- AdamW
 * For every element, with g = grad * *grad_scale and 32-bit arithmetic:
 *     m = beta1 m + (1 - beta1) g            v = beta2 v + (1 - beta2) g^2
 *     p = p (1 - lr weight_decay) - lr (m / (1 - beta1^step))
 *                                       / (sqrt(v / (1 - beta2^step)) + eps)
 * States of 32 bits are m and v as float32.  States of 8 bits are m and
 * sqrt(v), each as an 8-bit float (4 exponent bits with bias 7, 3 fraction
 * bits, the format with the largest value 448) times a power of two that the
 * LSTM_ADAMW_BLOCK elements of a block share:
 *     scale = 2^(E - 7), E the exponent of the block's largest magnitude
 * (at least 2^-126).  A value between two codes goes up or down by chance, in
 * proportion (nearest rounding would stand still, since one step changes v by
 * about a thousandth), with bits from a hash of the element's index in its
 * tensor and `seed`; sqrt(v) of a positive v is at least the smallest code.
 * What is not finite does not count for the scale and is stored as the format's
 * NaN; for sqrt(v) that NaN is read as infinity, so that an element whose g^2
 * left the fp32 range keeps its step of 0, as with states of 32 bits.
 * The update of p uses m and v before they are stored.  A bf16 parameter with
 * a float32 master copy is updated there and stored as its rounding. */
#define LSTM_ADAMW_BLOCK 256

typedef struct {
    void *param;        /* [n] dtype, updated */
    const void *grad;   /* [n] dtype */
    void *m, *v;        /* [n] float32, or [n] 8-bit codes; updated */
    float *m_scale, *v_scale; /* 8 bits: [ceil(n / LSTM_ADAMW_BLOCK)] each; 32 bits: not read */
    float *master;      /* [n] float32, updated, or NULL; bf16 parameters only */
    long long n;        /* >= 0 */
    float lr, weight_decay;
} lstm_adamw_tensor;

/* tensors: HOST array of count entries (read before the call returns).
 * state_bits 8 or 32; beta1, beta2 in [0, 1); eps >= 0; step >= 1;
 * grad_scale: one float32 in device memory (read by the kernels, so a
 * clipping factor needs no host wait), or NULL (1). */
lstm_status lstm_adamw_step(int dtype, int state_bits, const lstm_adamw_tensor *tensors, int count, double beta1,
                            double beta2, double eps, long long step, const float *grad_scale, unsigned seed,
                            void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LSTM_AMD_LSTM_OPS_H */
