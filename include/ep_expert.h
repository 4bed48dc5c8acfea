/*
 * ep_expert.h - the experts' products for prompts, decode batches and training,
 * for AMD Instinct MI355X (gfx950); part of the same library as ep.h (libep.so).
 *
 * ep_layer.h has the experts' products with 4-bit weights.  Here are those with
 * 8-bit integers, for serving, and the gated feed-forward block in bf16 with its
 * gradients, for training and serving:
 *   ep_quantize_i8, ep_quantize_i8_rows  rows in 8-bit integers, one scale a row
 *   ep_expert_i8             every expert's rows times its int8 weights, with the
 *                            gated activation on the way out where that is wanted
 *   ep_expert_ffn            gate and up projections with the activation, and the
 *                            product back down
 *   ep_expert_ffn_backward   its gradients: of the rows, both weights and the row
 *                            weights
 * A layer that serves in 8 bits runs
 *   ep_quantize_i8 -> ep_layout -> ep_expert_i8 (gated, the tokens' own rows) ->
 *   ep_quantize_i8_rows -> ep_expert_i8 -> ep_combine;
 * one that trains
 *   ep_layout -> ep_dispatch -> ep_expert_ffn -> ep_combine, and
 *   ep_combine_backward -> ep_expert_ffn_backward -> ep_dispatch_backward.
 *
 * Memory, streams, errors and graph capture are as in ep.h and ep_layer.h: nothing
 * here allocates, synchronises or keeps a pointer; a call enqueues on `stream`;
 * what the host can see is checked before anything is launched.  Calls on expert
 * rows take a handle that has been laid out, touch only rows that hold a slot, and
 * do nothing after a capacity or timeout error on the handle.  An output overlaps no
 * input and no other output but where it is said that it may be one
 * (EP_ERR_UNSUPPORTED).  Weights are as a model's file has them: no
 * packing.  bf16 rounding is to nearest, ties to even.  The order of all sums
 * depends on the sizes and the layout alone.  ep_time_next_call does not apply.
 */
#ifndef EP_EXPERT_H
#define EP_EXPERT_H

#include "ep.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * s = max(max_c |x[r][c]|, 1e-12) / 127,  q[r][c] = rint(x[r][c] / s), both divisions
 * in binary32, rounded once; ties go to the even code.  A row that holds a NaN or
 * an infinity gets the scale NaN and codes 0, so whatever is made of it is NaN.
 *   x          device bf16 [num_rows, channels] (ep_quantize_i8) or
 *              [capacity, channels], of which the rows that hold a slot count
 *              (ep_quantize_i8_rows).  channels % 16 == 0, channels <= 32768;
 *              16-byte aligned.
 *   out_q      device int8 of the same shape, 16-byte aligned.
 *   out_scale  device fp32 [num_rows] or [capacity].
 * With num_rows 0 the pointers may be NULL.
 */
ep_status ep_quantize_i8(const void *x, int32_t num_rows, int32_t channels, void *out_q,
                         float *out_scale, hipStream_t stream);
ep_status ep_quantize_i8_rows(const ep_handle *h, const void *x, int32_t channels, void *out_q,
                              float *out_scale, hipStream_t stream);

/*
 * v[r][j] = float(sum_c x[r][c] * w[e][j][c]) * x_scale[r] * w_scale[e][j]
 * for every expert e and every row r of its segment; the sum is exact (32-bit
 * integers), the rest binary32.  out[r] = bf16(v[r]), or with `gated`, the rows of
 * w[e] being n/2 of gate and then n/2 of up,
 *   out[r][i] = bf16(silu(v[r][i]) * v[r][n/2 + i] * row_weights[r]),
 * silu as in ep_swiglu.
 *   x        device int8 rows of k channels, 16-byte aligned; k % 16 == 0, k <= 32768.
 *   x_scale  device fp32, one a row of x.
 *   token_rows  0: x is [capacity, k], expanded rows as dispatch writes them.
 *            1: x is [num_tokens, k] and an expanded row reads its slot's token.
 *   w        device int8 [E, n, k], 16-byte aligned; n % 8 == 0 (gated: n % 16 == 0),
 *            n <= 65536.
 *   w_scale  device fp32 [E, n], 16-byte aligned.
 *   row_weights  NULL (weight 1) or, gated, fp32 [capacity].
 *   out      device bf16 [capacity, n] (gated: [capacity, n/2]), 16-byte aligned.
 */
ep_status ep_expert_i8(const ep_handle *h, const void *x, const float *x_scale,
                       int32_t token_rows, int32_t k, const void *w, const float *w_scale,
                       int32_t n, int32_t gated, const float *row_weights, void *out,
                       hipStream_t stream);

/*
 * The experts' gated feed-forward block, for every expert e and every row r of its
 * segment, sums in binary32:
 *   gate_up[r] = w13[e] . x[r]        (inter rows of gate, then inter of up)
 *   h[r] = bf16(silu(gate) * up * row_weights[r])
 *   y[r] = bf16(w2[e] . h[r])
 * in two launches: h is made from the binary32 sums, gate_up goes to memory only
 * where it is wanted.
 *   x        device bf16 [capacity, hidden], or with token_rows 1 [num_tokens, hidden]
 *            (an expanded row reads its slot's token).
 *   w13      device bf16 [E, 2 inter, hidden];  w2  device bf16 [E, hidden, inter].
 *            hidden % 8 == 0, inter % 8 == 0, both <= 32768.
 *   row_weights  NULL (weight 1) or fp32 [capacity], as dispatch's out_w.
 *   out_h    device bf16 [capacity, inter].
 *   saved    NULL or bf16 [capacity, 2 inter]: gate_up, rounded, for the backward pass.
 *   out_y    device bf16 [capacity, hidden].  May be NULL together with w2: the
 *            projections and the activation alone.
 * All 16-byte aligned (row_weights 4).
 */
ep_status ep_expert_ffn(const ep_handle *h, const void *x, int32_t token_rows, int32_t hidden,
                        const void *w13, const void *w2, int32_t inter,
                        const float *row_weights, void *out_h, void *saved, void *out_y,
                        hipStream_t stream);

/*
 * Gradients of ep_expert_ffn for gy = d loss / d y, with s = 1 / (1 + exp(-gate)) and
 * w = row_weights[r], gate and up the values in `saved`:
 *   gh = gy . w2[e]                               (binary32, not stored)
 *   grad_gate = bf16(w gh up s (1 + gate (1 - s))),  grad_up = bf16(w gh gate s)
 *   grad_row_weights[r] = sum_i gh gate s up
 *   grad_x[r] = bf16(grad_gate_up[r] . w13[e])
 *   grad_w13[e] = sum_r grad_gate_up[r] x[r]^T,   grad_w2[e] = sum_r gy[r] h[r]^T
 * (zeros for an expert without rows).
 *   grad_y   device bf16 [capacity, hidden].
 *   x        as in the forward pass; needed for grad_w13.
 *   saved    device bf16 [capacity, 2 inter].
 *   rows_h   device bf16 [capacity, inter]: the forward's h, needed for grad_w2; with
 *            remake_h 1 it is written, from `saved`, and may be any buffer.
 *   grad_gate_up  device bf16 [capacity, 2 inter], written; may be `saved` itself.
 *   grad_x   NULL or bf16 [capacity, hidden], the gradient of the expanded rows
 *            (ep_dispatch_backward sums them into tokens); w13 may be NULL without it.
 *   grad_w13, grad_w2  NULL or device, the shapes of w13 and w2, in grad_dtype:
 *            EP_BF16 or EP_F32.
 *   grad_row_weights  NULL or fp32 [capacity].
 *   workspace  ep_expert_ffn_backward_workspace bytes, 16-byte aligned; only used
 *            with grad_row_weights, else it may be NULL.
 * All 16-byte aligned (row_weights and grad_row_weights 4).
 */
size_t ep_expert_ffn_backward_workspace(const ep_handle *h, int32_t inter);
ep_status ep_expert_ffn_backward(const ep_handle *h, const void *grad_y, const void *x,
                                 int32_t token_rows, int32_t hidden, const void *w13,
                                 const void *w2, int32_t inter, const float *row_weights,
                                 const void *saved, void *rows_h, int32_t remake_h,
                                 void *grad_gate_up, void *grad_x, ep_dtype grad_dtype,
                                 void *grad_w13, void *grad_w2, float *grad_row_weights,
                                 void *workspace, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EP_EXPERT_H */
