/*
 * moe_train.h -- C ABI of the expert layer in bf16 with its gradients, part of
 * libmoe_dispatch.so: the experts' products for rows and weights in bf16, what
 * their epilogues do, and every gradient of a layer between dispatch and
 * combine.
 *
 *   moe_ffn_gated            gate and up products, activation, product
 *   moe_expert_linear        product with bias, activation and residual
 *   moe_activation_backward  gradients of both, before their products
 *   moe_expert_grad_input    gradient of a product to its rows
 *   moe_expert_grad_weight   gradient of a product to its weights and bias
 *   moe_combine_backward     gradient of moe_combine
 *
 * A layer's step, rows in the dispatched layout (moe_dispatch, quant NONE):
 *   forward   moe_dispatch -> a;  moe_ffn_gated(a, w13) -> h, saved;
 *             moe_expert_linear(h, w2) -> y;  moe_combine(y, topk_w) -> out
 *   backward  moe_combine_backward(dout, y) -> dy, dtopk_w;
 *             moe_expert_grad_input(dy, w2) -> dh;
 *             moe_activation_backward(dh, saved) -> dsaved, h;
 *             moe_expert_grad_weight(dy, h) -> dw2;
 *             moe_expert_grad_input(dsaved, w13) -> da;
 *             moe_expert_grad_weight(dsaved, a) -> dw13;
 *             moe_combine with every weight 1 (da) -> dx: dispatch's gradient
 * so h is not kept, and `saved` and a may be kept in 8 bits.
 *
 * The conventions of moe_dispatch.h hold: device pointers owned by the caller,
 * dense row-major arrays, no allocation, no synchronization, no state kept
 * between calls, argument errors returned before anything is enqueued, work
 * enqueued on `stream` and capturable in a HIP graph.  Results do not depend on
 * timing: no sum's order is left to the scheduling.
 *
 * Rows are those of the dispatch that `handle` describes, or, with a NULL
 * handle, the num_tokens rows of one dense group (cfg.num_experts must be 1).
 * rows = moe_rows_capacity(cfg), or num_tokens.  Rows that hold no pair are
 * neither read nor written.  num_tokens is the batch of the dispatch: it sizes
 * launches, so the handle must hold at most num_tokens * K pairs.  cfg.quant and
 * (but where it is named) cfg.hidden are not used.
 *
 * Arrays are bf16 bits unless said otherwise, 16-byte aligned (scales, biases'
 * gradients and topk_w 4).  Outputs must not overlap other arguments except where
 * that is said.  Channel counts are multiples of 8 and at most
 * MOE_TRAIN_MAX_CHANNELS (larger: MOE_ERR_UNSUPPORTED).  Sums are fp32, every
 * output is rounded once.  A sum with a NaN is NaN, an infinite value gives what
 * the formula gives; no row shows in another's result.
 *
 * Saved rows.  The input of an activation can be kept for its gradient, in
 * saved_quant's format: MOE_QUANT_NONE, bf16 rows (saved_scale NULL), or E4M3
 * rows with scales as moe_dispatch writes them (channels then a multiple of 128).
 * Scales follow the fp32 sums: a block whose largest value lies within their error of
 * a format's border (448 times a power of two) may take the scale on either side.
 */
#ifndef MOE_TRAIN_H
#define MOE_TRAIN_H

#include "moe_dispatch.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_TRAIN_MAX_CHANNELS (1 << 20)

/* Activations. */
#define MOE_ACT_NONE 0
#define MOE_ACT_SILU 1 /* v / (1 + exp(-v)) */
#define MOE_ACT_GELU 2 /* v / 2 (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))) */
#define MOE_ACT_RELU 3 /* v > 0 ? v : 0 (slope 0 at 0) */
/* Where 1 / (1 + exp(-z)) is below 2^-126 (z = v for SiLU, sqrt(8/pi) (v + 0.044715 v^3)
 * for GELU; v < -87.3 and v < -10) both and their slopes are 0. */

/*
 * The gated block: for every row of expert e, with p = a . w13[e] and g, u its
 * channels [0, inter) and [inter, 2 * inter),
 *   h = bf16( act(g) * u ),  saved = p.
 *
 *   a            [rows, cfg.hidden].
 *   w13          [E, 2 * inter, cfg.hidden], gate channels first.
 *   h            [rows, inter].
 *   saved        [rows, 2 * inter] or NULL (saved_scale NULL too).
 * 8-bit saved rows need inter to be a multiple of 128.
 */
moe_status_t moe_ffn_gated(const moe_config_t *cfg, int32_t num_tokens, int32_t inter, int32_t act,
                           const uint16_t *a, const uint16_t *w13, const moe_handle_t *handle, uint16_t *h,
                           void *saved, void *saved_scale, int32_t saved_quant, void *stream);

/*
 * A product with its epilogue: with p = a . w[e] + bias[e],
 *   y = bf16( act(p) + residual ),  saved = p.
 *
 *   n, k         output and input channels.
 *   a            [rows, k].
 *   w            [E, n, k].
 *   bias         [E, n] or NULL.
 *   residual     [rows, n] or NULL; may be y's array.
 *   y            [rows, n].
 *   saved        [rows, n] or NULL (saved_scale NULL too).
 */
moe_status_t moe_expert_linear(const moe_config_t *cfg, int32_t num_tokens, int32_t n, int32_t k, int32_t act,
                               const uint16_t *a, const uint16_t *w, const uint16_t *bias, const uint16_t *residual,
                               const moe_handle_t *handle, uint16_t *y, void *saved, void *saved_scale,
                               int32_t saved_quant, void *stream);

/*
 * Gradients of an activation from its saved input, and its output again.
 * Gated (saved = g, u of n channels each):
 *   dsaved = bf16( dy * u * act'(g) ), bf16( dy * act(g) ),  y = bf16( act(g) * u )
 * else
 *   dsaved = bf16( dy * act'(saved) ),  y = bf16( act(saved) ).
 *
 *   n            channels of dy.
 *   gated        0 or 1.
 *   dy           [rows, n].
 *   saved        [rows, 2 * n] or [rows, n] in saved_quant's format, saved_scale
 *                its scales.
 *   dsaved       [rows, 2 * n] or [rows, n]; may be saved's array (bf16).
 *   y            [rows, n] or NULL; may be dy's array.
 */
moe_status_t moe_activation_backward(const moe_config_t *cfg, int32_t num_tokens, int32_t n, int32_t act,
                                     int32_t gated, const uint16_t *dy, const void *saved, const void *saved_scale,
                                     int32_t saved_quant, const moe_handle_t *handle, uint16_t *dsaved, uint16_t *y,
                                     void *stream);

/*
 * Gradient of p = a . w[e] to a:  da[row, c] = bf16( sum over j of dy[row, j] *
 * w[e, j, c] ).
 *
 *   dy           [rows, n].
 *   w            [E, n, k].
 *   da           [rows, k].
 */
moe_status_t moe_expert_grad_input(const moe_config_t *cfg, int32_t num_tokens, int32_t n, int32_t k,
                                   const uint16_t *dy, const uint16_t *w, const moe_handle_t *handle, uint16_t *da,
                                   void *stream);

/*
 * Gradients of p = a . w[e] + bias[e] to w and bias:
 *   dw[e, j, c] = sum over rows of e of dy[row, j] * a[row, c],
 *   dbias[e, j] = sum over rows of e of dy[row, j].
 * Experts without rows get zeros (or, with accumulate, keep what they have).
 *
 *   dy           [rows, n].
 *   a            [rows, k] in a_quant's format (MOE_QUANT_NONE: bf16, a_scale
 *                NULL; else E4M3 with a_scale as moe_dispatch writes them, k a
 *                multiple of 128).  8-bit rows count as the bf16 values nearest to
 *                value * scale (exact for UE8M0 and MXFP8 within bf16's range).
 *   dw           fp32 or (dw_bf16 != 0) bf16 [E, n, k].
 *   dbias        fp32 [E, n] or NULL.
 *   accumulate   1: dw (fp32 only) and dbias are added to; 0: written.
 *   workspace    >= moe_grad_weight_workspace_bytes bytes, 16-byte aligned,
 *                clobbered: two calls that may overlap need one each.  NULL if
 *                that is 0.
 */
moe_status_t moe_expert_grad_weight(const moe_config_t *cfg, int32_t num_tokens, int32_t n, int32_t k,
                                    const uint16_t *dy, const void *a, const void *a_scale, int32_t a_quant,
                                    const moe_handle_t *handle, void *dw, int32_t dw_bf16, float *dbias,
                                    int32_t accumulate, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of device workspace moe_expert_grad_weight needs for num_tokens tokens on
 * the current device (few weights share their rows' sums among more of the chip
 * and join them there; 0 for most sizes).  0 for arguments that it refuses. */
size_t moe_grad_weight_workspace_bytes(const moe_config_t *cfg, int32_t num_tokens, int32_t n, int32_t k);

/*
 * Gradient of moe_combine: for every kept pair p = t * K + j, row =
 * pair_to_row[p],
 *   dy[row] = bf16( topk_w[p] * dout[t] ),  dtopk_w[p] = sum over c of dout[t, c] * y[row, c];
 * dtopk_w is 0 for pairs that are not kept (their weight is not read).
 *
 *   dout         [num_tokens, cfg.hidden].
 *   y            [rows, cfg.hidden], combine's input; NULL if dtopk_w is NULL.
 *   topk_w       fp32 [num_tokens, K].
 *   handle       of the dispatch; not NULL.
 *   dy           [rows, cfg.hidden]; may be y's array.
 *   dtopk_w      fp32 [num_tokens, K] or NULL.
 */
moe_status_t moe_combine_backward(const moe_config_t *cfg, int32_t num_tokens, const uint16_t *dout,
                                  const uint16_t *y, const float *topk_w, const moe_handle_t *handle, uint16_t *dy,
                                  float *dtopk_w, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_TRAIN_H */
