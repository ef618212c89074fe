/*
 * lstm_blocks.h -- operators that make blocks of a sequence model out of the
 * layers of lstm.h and the operators of lstm_ops.h: a gated linear recurrence
 * (a recurrent layer whose gates come from its input alone, so that time need
 * not be walked step by step), rotary positions with the norm of each head
 * (in front of linear attention), and the gated feed-forward block.
 *
 * Conventions are those of lstm_ops.h: device memory of the current device,
 * owned by the caller; scratch in a caller's workspace whose size a query
 * gives; a stream argument (NULL = default stream); an lstm_status from every
 * call; host checks before anything is enqueued; no exception crosses the
 * interface; nothing is allocated.  Calls may be captured into a graph; two
 * calls that may run at once need workspaces of their own.  Dtypes: LSTM_F32
 * and LSTM_BF16.  Sums, states and statistics are fp32 and so is all
 * arithmetic, but for the angles (64 bits) and the bf16 operands of the
 * feed-forward block's products (see there).
 */
#ifndef LSTM_AMD_LSTM_BLOCKS_H
#define LSTM_AMD_LSTM_BLOCKS_H

#include <stddef.h>

#include "lstm_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------- gated linear recurrence
 * For every channel, with s(.) the logistic function, forget and input gate
 * as given before it (their logits f and i), and a state h:
 *     a_t = s(f_t)        w_t = s(i_t), or 1 - a_t without an input gate
 *     h_t = a_t h_{t-1} + w_t x_t         y_t = h_t
 * computed from the smaller of a_t and 1 - a_t = s(-f_t), so that gates keep
 * their digits near 0 and near 1 (gates below 2^-126 are 0).  An infinite
 * state stays infinite, past a gate of 0, too. */
typedef struct {
    int dtype;  /* lstm_dtype of x, the gates, y and their gradients */
    int T, B;   /* >= 1; T at most 2^30 */
    int width;  /* channels, 1..2^20 */
} lstm_gated_recurrence_shape;

/* Bytes of workspace (0 is possible) of the forward and of the backward call
 * of this shape.  Touches no device. */
lstm_status lstm_gated_recurrence_workspace_size(const lstm_gated_recurrence_shape *shape, size_t *bytes);
lstm_status lstm_gated_recurrence_backward_workspace_size(const lstm_gated_recurrence_shape *shape, size_t *bytes);

/* Whole sequences.
 *   x, forget, input  [T, B, width] views (lstm_ops.h; the head stride is not
 *                used): any strides and any alignment.  input: NULL for w = 1 - a
 *   lengths      [B] int32 DEVICE memory, or NULL (every row has T tokens);
 *                values are clamped to 0..T.  Tokens past a row's length are
 *                not read, their y is 0, and the row's state passes them by.
 *   state        [B, width] float32, the state before the first token, or
 *                NULL (zeros)
 *   y            view, written; must not overlap an input or itself
 *   state_out    like state: the state after each row's last token, or NULL.
 *                It may be the memory of `state`.
 *   workspace    16-byte aligned.  Where it has bytes, workgroups wait for
 *                each other through it.  A wait ends after five seconds at the
 *                latest, as it can where two calls at once share a workspace:
 *                what depends on it is NaN then.
 * LSTM_ERR_ARG: NULL argument; LSTM_ERR_SHAPE: T, B or width outside their
 * limits, or B * width above 2^31 - 1; LSTM_ERR_WORKSPACE: workspace too short. */
lstm_status lstm_gated_recurrence_forward(const lstm_gated_recurrence_shape *shape, const lstm_view *x,
                                          const lstm_view *forget, const lstm_view *input, const int *lengths,
                                          const float *state, const lstm_view *y, float *state_out, void *workspace,
                                          size_t workspace_bytes, void *stream);

/* Gradients of that forward.  y: as the forward wrote it (bf16: h_{t-1} is
 * read from there with its rounding; the gradient of `forget` is off by that);
 * dy: gradient of y; dstate_out: gradient of state_out, or NULL (zeros); dx,
 * dforget, dinput: views, written (dinput NULL exactly where input is);
 * dstate: gradient of state, or NULL.  Tokens past a row's length get zero
 * gradients.  Outputs must not overlap inputs. */
lstm_status lstm_gated_recurrence_backward(const lstm_gated_recurrence_shape *shape, const lstm_view *x,
                                           const lstm_view *forget, const lstm_view *input, const int *lengths,
                                           const float *state, const lstm_view *y, const lstm_view *dy,
                                           const float *dstate_out, const lstm_view *dx, const lstm_view *dforget,
                                           const lstm_view *dinput, float *dstate, void *workspace,
                                           size_t workspace_bytes, void *stream);

/* One token for each of B requests (shape->T must be 1; the views' time
 * strides are not used).  pool [n_slots, width] float32 holds the requests'
 * states and is updated in place.
 *   slots  [B] int32 device memory: row b's state is pool[slots[b]]; a value
 *          outside 0..n_slots-1 marks an idle row, whose y is 0.  Two rows of
 *          one call must not name the same slot.  NULL: row b uses slot b
 *          (n_slots >= B, else LSTM_ERR_SHAPE). */
lstm_status lstm_gated_recurrence_step(const lstm_gated_recurrence_shape *shape, const lstm_view *x,
                                       const lstm_view *forget, const lstm_view *input, const int *slots, int n_slots,
                                       float *pool, const lstm_view *y, void *stream);

/* --------------------------------------------------------------------- rotary
 * Queries and keys of a layer, head by head: the norm of the head, then the
 * rotation of its first rotary_dim values by the token's position p.
 *     u = x weight / sqrt(mean(x^2) + eps)   (norm 0: u = x; the squares are
 *                                             summed in fp32)
 *     (u_a, u_b) -> m (u_a cos(p f_j) - u_b sin(p f_j), u_b cos + u_a sin)
 * for the pairs j = 0 .. rotary_dim / 2 - 1, (a, b) = (j, j + rotary_dim / 2),
 * or (2j, 2j + 1) where interleaved.  Values past rotary_dim are not turned. */
typedef struct {
    int dtype;            /* lstm_dtype of q, k, the weights and all gradients */
    int T, B;             /* >= 1; T * B at most 2^31 - 1 */
    int heads, kv_heads;  /* heads >= 1, kv_heads >= 0 (0: no keys); each at most 2^16 */
    int dim;              /* of a head, 1..256 */
    int rotary_dim;       /* 0..dim, even */
    int interleaved;      /* 0 or 1 */
    int norm;             /* 0 or 1 */
    float eps;            /* >= 0 and finite */
    float scale;          /* m, finite (1: rotation alone) */
} lstm_rotary_shape;

/* Positions of the tokens: int32 device memory with the element strides of
 * time and batch (0 repeats), any values; data NULL: token t stands at t. */
typedef struct {
    const int *data;
    long long time, batch;
} lstm_positions;

/* q, k: views of [T, B, heads, dim] and [T, B, kv_heads, dim], any strides and
 * alignment, the last axis dense.  q_weight, k_weight: [dim], or NULL (ones);
 * with norm 0 both must be NULL.  frequencies: [rotary_dim / 2] float64 device
 * memory, radians a position (NULL for rotary_dim 0).  q_out, k_out: views,
 * written; each may be its input's memory with the same strides, and must not
 * overlap anything else.  The k arguments are not read with kv_heads 0.
 * positions: NULL as one whose data is NULL. */
lstm_status lstm_rotary_forward(const lstm_rotary_shape *shape, const lstm_view *q, const lstm_view *k,
                                const void *q_weight, const void *k_weight, const double *frequencies,
                                const lstm_positions *positions, const lstm_view *q_out, const lstm_view *k_out,
                                void *stream);

lstm_status lstm_rotary_backward_workspace_size(const lstm_rotary_shape *shape, size_t *bytes);

/* Gradients.  q, k: the forward's inputs (read only where norm is 1: else they
 * may be NULL); dq_out, dk_out: gradients of its outputs; dq, dk: views,
 * written; each may be the memory of its output's gradient with the same
 * strides.  dq_weight, dk_weight: [dim] dtype, or NULL (not wanted; with norm 0
 * they must be); summed over tokens and heads in a fixed order. */
lstm_status lstm_rotary_backward(const lstm_rotary_shape *shape, const lstm_view *q, const lstm_view *k,
                                 const void *q_weight, const void *k_weight, const double *frequencies,
                                 const lstm_positions *positions, const lstm_view *dq_out, const lstm_view *dk_out,
                                 const lstm_view *dq, const lstm_view *dk, void *dq_weight, void *dk_weight,
                                 void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------ gated MLP
 *     g = x w_gate^T    u = x w_up^T    h = act(g) u    y = h w_down^T
 * The products run on the matrix cores and are summed in fp32.  LSTM_BF16: h
 * and, in the backward call, the kept g and u and the gradients of g and u are
 * rounded as operands, each once (h and the gradients to 8 bits; g and u are
 * kept with 16).  LSTM_F32: every operand is split into three bf16 terms, whose
 * six largest products are summed (2^-24 of each operand; values below 2^-100
 * keep fewer bits); a value that is not finite spoils the outputs it reaches,
 * as NaN.  Up to 64 rows of a forward call are multiplied in fp32 itself. */
typedef enum {
    LSTM_ACT_SILU = 0,    /* g s(g) */
    LSTM_ACT_GELU = 1,    /* g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2 */
    LSTM_ACT_SIGMOID = 2  /* s(g) */
} lstm_activation;

typedef struct {
    int dtype;
    int activation;        /* lstm_activation */
    int rows;              /* tokens, 0..2^30; times the widest of the others at most 2^38 */
    int in, hidden, out;   /* 1..2^18 */
} lstm_gated_mlp_shape;

lstm_status lstm_gated_mlp_workspace_size(const lstm_gated_mlp_shape *shape, size_t *bytes);
lstm_status lstm_gated_mlp_reserve_size(const lstm_gated_mlp_shape *shape, size_t *bytes);
lstm_status lstm_gated_mlp_backward_workspace_size(const lstm_gated_mlp_shape *shape, size_t *bytes);

/* x [rows, in], rows x_stride >= in elements apart; w_gate, w_up [hidden, in],
 * w_down [out, hidden], y [rows, out]: dense.  reserve: NULL, or memory of
 * lstm_gated_mlp_reserve_size bytes that receives g, u and h for the backward
 * call (16-byte aligned, as the workspace).  rows 0 does nothing.  y must not
 * overlap an input. */
lstm_status lstm_gated_mlp_forward(const lstm_gated_mlp_shape *shape, const void *x, long long x_stride,
                                   const void *w_gate, const void *w_up, const void *w_down, void *y, void *reserve,
                                   size_t reserve_bytes, void *workspace, size_t workspace_bytes, void *stream);

/* Gradients.  reserve: as the forward with the same arguments wrote it, not
 * changed; dy [rows, out], rows dy_stride apart; dx [rows, in], dw_gate, dw_up
 * [hidden, in], dw_down [out, hidden]: dense, written, each may be NULL (not
 * wanted).  rows 0: the weights' gradients are zeros.  Sums run in a fixed
 * order. */
lstm_status lstm_gated_mlp_backward(const lstm_gated_mlp_shape *shape, const void *x, long long x_stride,
                                    const void *w_gate, const void *w_up, const void *w_down, const void *reserve,
                                    size_t reserve_bytes, const void *dy, long long dy_stride, void *dx, void *dw_gate,
                                    void *dw_up, void *dw_down, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LSTM_AMD_LSTM_BLOCKS_H */
