/*
 * ep_layer.h - operators of the expert layer around dispatch and combine, for
 * AMD Instinct MI355X (gfx950); part of the same library as ep.h (libep.so).
 *
 * A mixture-of-experts layer runs
 *   add + norm (FP8 out) -> layout -> dispatch -> product with the experts'
 *   4-bit weights -> gated activation -> product -> combine
 * when it serves, and
 *   add + norm -> layout -> dispatch -> caller's grouped GEMM -> gated
 *   activation with an 8-bit checkpoint -> caller's grouped GEMM -> combine
 * and back again when it trains.  ep.h has layout, dispatch, combine and the
 * gradients of the last two; this header has the steps between:
 *   ep_add_rmsnorm           sum with the residual, root-mean-square norm, rows
 *                            in bf16 and / or E4M3 with scales
 *   ep_add_rmsnorm_backward  its gradients
 *   ep_expert_w4             every expert's rows times its 4-bit weights
 *   ep_swiglu                silu(gate) * up of the expert rows, in bf16 or E4M3,
 *                            with an E4M3 checkpoint of gate and up
 *   ep_swiglu_backward       its gradients, from that checkpoint
 *
 * Memory, streams, errors and graph capture are as in ep.h: nothing here
 * allocates, synchronises or keeps a pointer; a call enqueues on `stream`;
 * what the host can see is checked before anything is launched.  The calls
 * on expert rows take a handle that has been laid out (ep.h), touch only
 * rows that hold a slot (gap rows and rows at or past psum[E] are neither
 * read nor written) and, like dispatch, do nothing after a capacity or
 * timeout error on the handle.  An output overlaps no input and no other output
 * but where it is said that it may be one (of the row buffers such calls are refused with
 * EP_ERR_UNSUPPORTED).  bf16 rounding is to nearest, ties to even.
 * ep_time_next_call does not apply to these calls.
 *
 * E4M3 rows ("codes") and their scales are those of ep_quantize_fp8: blocks of
 * 128 channels, s = max(amax, 1e-12) / 448, EP_SF_F32 or EP_SF_UE8M0 packs
 * with a token stride and a pack stride.  Below, "sf" arguments are
 * (pointer, token stride, pack stride) in 4-byte packs, ep_sf_packs() a row.
 */
#ifndef EP_LAYER_H
#define EP_LAYER_H

#include "ep.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * z = bf16(x + residual) (z = x without a residual)
 * rstd = 1 / sqrt(mean(z^2) + eps), the mean over the row's `hidden` channels
 * y = (z * rstd) * weight
 * The squares are summed in binary64 and rstd is rounded once to binary32, so
 * the rows do not depend on the order of the sum; y is two binary32 products.
 *   x, residual  device bf16 [num_tokens, hidden]; residual may be NULL.
 *                hidden % 8 == 0, hidden <= 32768; 16-byte aligned.
 *   weight       device [hidden], EP_BF16 or EP_F32; 16-byte aligned.
 *   eps          finite, >= 0.
 *   out_z        NULL or bf16 [num_tokens, hidden]; may be x or residual itself.
 *   out_y        NULL or bf16 [num_tokens, hidden]: y rounded once.
 *   out_q        NULL or E4M3 codes [num_tokens, hidden] of y as it is in
 *                binary32 (not of the bf16 y), hidden % 128 == 0, with scales
 *                out_sf in format fmt.
 *   out_rstd     NULL or fp32 [num_tokens], for the backward pass.
 * At least one output is needed.  With num_tokens 0 every pointer may be NULL.
 */
ep_status ep_add_rmsnorm(const void *x, const void *residual, const void *weight,
                         ep_dtype weight_dtype, float eps, int32_t num_tokens, int32_t hidden,
                         void *out_z, void *out_y, ep_sf_format fmt, void *out_q, void *out_sf,
                         int64_t out_sf_token_stride, int64_t out_sf_hidden_stride,
                         float *out_rstd, hipStream_t stream);

/*
 * Gradients of ep_add_rmsnorm, from the saved z and rstd.  With n = z * rstd and
 * g = d loss / d y (an E4M3 output's gradient is taken as y's):
 *   c[t] = mean_h(g * weight * n)
 *   grad_x      = rstd * (g * weight - n * c) + grad_z
 *   grad_weight = sum_t g * n
 *   grad_y, z   device bf16 [num_tokens, hidden], as above.
 *   grad_z      NULL or bf16 [num_tokens, hidden]: the gradient that reaches z
 *               on its other way, along the residual.
 *   grad_x      NULL or bf16 [num_tokens, hidden]: gradient of x and of the
 *               residual (they share it); may be grad_y, grad_z or z itself.
 *   grad_weight NULL or fp32 [hidden], summed in binary32 in a fixed order
 *               (zeros when num_tokens is 0).
 *   workspace   device, 16-byte aligned, ep_add_rmsnorm_backward_workspace bytes;
 *               may be NULL without grad_weight, and where that function gives 0: for
 *               few rows (and for invalid sizes).
 */
size_t ep_add_rmsnorm_backward_workspace(int32_t num_tokens, int32_t hidden);
ep_status ep_add_rmsnorm_backward(const void *grad_y, const void *z, const void *weight,
                                  ep_dtype weight_dtype, const float *rstd, const void *grad_z,
                                  int32_t num_tokens, int32_t hidden, void *grad_x,
                                  float *grad_weight, void *workspace, size_t ws_bytes,
                                  hipStream_t stream);

/*
 * 4-bit weights of the experts, W[e] = [n, k], scaled in groups of `group`
 * consecutive channels of k.
 */
typedef enum ep_w4_format {
    EP_W4_INT4 = 0,           /* value (code - 8) * scale, code 0..15, bf16       */
                              /* scales, group 32, 64 or 128                      */
    EP_W4_MXFP4 = 1           /* E2M1 code * 2^(byte - 127), group 32: byte 0 is  */
                              /* 2^-127, a weight of 2^128 or more (bytes 253 and */
                              /* 254) infinite; byte 255 makes the group NaN      */
} ep_w4_format;

/*
 * Lays weights out for ep_expert_w4, once, when a model is loaded.
 *   codes   device uint8 [E, n, k/2]: channel 2j in the low half of byte j.
 *   scales  device [E, n, k/group]: bf16 (EP_W4_INT4) or uint8 (EP_W4_MXFP4).
 *   out_codes, out_scales  device, 16-byte aligned, ep_w4_code_bytes /
 *           ep_w4_scale_bytes bytes (0 if the sizes are invalid).
 * 1 <= E <= 1024, n % 8 == 0, k % 128 == 0, k <= 32768.
 */
size_t ep_w4_code_bytes(int32_t num_experts, int32_t n, int32_t k);
size_t ep_w4_scale_bytes(int32_t num_experts, int32_t n, int32_t k, ep_w4_format fmt,
                         int32_t group);
ep_status ep_w4_pack(const void *codes, const void *scales, int32_t num_experts, int32_t n,
                     int32_t k, ep_w4_format fmt, int32_t group, void *out_codes,
                     void *out_scales, hipStream_t stream);

/*
 * out[r] = bf16(W[e] . x[r]) for every expert e and every row r of its segment
 * that holds a slot: the experts' products for decode batches, where each
 * expert has few rows and the weights are what is read.  Products and sums
 * are binary32, one rounding at the end.
 *   x       device rows of k channels, 16-byte aligned: EP_BF16, or EP_FP8_E4M3
 *           codes with scales sf in format sf_fmt.
 *   token_rows  0: x (and sf) is [capacity, k], expanded rows as dispatch
 *           writes them.  1: x is [num_tokens, k] and an expanded row reads its
 *           slot's token, so a decode step needs no dispatch in front of it.
 *   codes, scales  from ep_w4_pack, for the handle's num_experts.
 *   out     device bf16 [capacity, n], 16-byte aligned; combine reads it.
 * The order of the sums depends on the sizes alone.  EP_W4_INT4 sums
 * (128 + code) x - 136 x, partial sums up to 136 times a group's sum of |x|: where
 * one leaves binary32 (bf16 rows with a group's sum of |x| above 2^120.9) the row's
 * outputs are infinite, of either sign, or NaN; a row that holds an infinity
 * comes out as NaN.
 */
ep_status ep_expert_w4(const ep_handle *h, const void *x, ep_dtype x_dtype, int32_t token_rows,
                       int32_t k, const void *sf, ep_sf_format sf_fmt, int64_t sf_token_stride,
                       int64_t sf_hidden_stride, const void *codes, const void *scales,
                       ep_w4_format fmt, int32_t group, int32_t n, void *out,
                       hipStream_t stream);

/*
 * Gated activation of the expert rows: with gate = gate_up[r][0 .. inter) and
 * up = gate_up[r][inter .. 2 inter),
 *   h = gate / (1 + exp(-gate)) * up * row_weights[r]
 * in binary32: for a gate below -87, where exp(-gate) nears the end of its range, the
 * quotient may come out as 0.
 *   gate_up     device bf16 [capacity, 2 inter], inter % 8 == 0,
 *               inter <= 32768, 16-byte aligned.
 *   row_weights NULL (weight 1) or fp32 [capacity], as dispatch's out_w.
 *   out_h       device [capacity, inter], 16-byte aligned: bf16, or with
 *               h_dtype EP_FP8_E4M3 codes of the binary32 h with scales out_sf
 *               in format fmt (inter % 128 == 0).
 *   saved       NULL or E4M3 codes [capacity, 2 inter] of gate_up with scales
 *               saved_sf in format saved_fmt (inter % 128 == 0): the checkpoint
 *               that ep_swiglu_backward reads in place of gate_up.
 */
ep_status ep_swiglu(const ep_handle *h, const void *gate_up, int32_t inter,
                    const float *row_weights, ep_dtype h_dtype, void *out_h, ep_sf_format fmt,
                    void *out_sf, int64_t out_sf_token_stride, int64_t out_sf_hidden_stride,
                    void *saved, ep_sf_format saved_fmt, void *saved_sf,
                    int64_t saved_sf_token_stride, int64_t saved_sf_hidden_stride,
                    hipStream_t stream);

/*
 * Gradients of ep_swiglu for g = d loss / d h (an E4M3 h's gradient is taken as
 * h's), with s = 1 / (1 + exp(-gate)):
 *   grad_gate = w * g * up * s * (1 + gate * (1 - s)),  grad_up = w * g * gate * s
 *   grad_row_weights[r] = sum_i g * gate * s * up  (binary32, fixed order)
 *   grad_h       device bf16 [capacity, inter].
 *   saved        device [capacity, 2 inter]: the bf16 gate_up itself
 *                (saved_dtype EP_BF16) or its checkpoint (EP_FP8_E4M3, with
 *                saved_sf; the gradient is that of the values it stands for).
 *   grad_gate_up device bf16 [capacity, 2 inter]; may be a bf16 `saved` itself.
 *   grad_row_weights  NULL or fp32 [capacity]; ep_dispatch_backward takes it.
 *   out_h        NULL or bf16 [capacity, inter]: h made again from `saved`, for
 *                the gradient of the weights that multiply it; may be grad_h
 *                itself.
 */
ep_status ep_swiglu_backward(const ep_handle *h, const void *grad_h, int32_t inter,
                             const float *row_weights, const void *saved, ep_dtype saved_dtype,
                             ep_sf_format saved_fmt, const void *saved_sf,
                             int64_t saved_sf_token_stride, int64_t saved_sf_hidden_stride,
                             void *grad_gate_up, float *grad_row_weights, void *out_h,
                             hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EP_LAYER_H */
