/*
 * moe_experts.h -- C ABI of the expert-layer operators of libmoe_dispatch.so:
 * what runs before, between and instead of the dispatch and combine calls of
 * moe_dispatch.h.
 *
 *   moe_rmsnorm             residual add + root-mean-square norm, with the
 *                           normed rows also in 8 bits (the dispatch's formats)
 *   moe_expert_gemm         the experts' products on dispatched FP8 rows
 *   moe_expert_gemm_swiglu  gate and up products, SwiGLU and requantization
 *   moe_layer_fused         a whole expert layer for at most 64 tokens
 *
 * A layer for prefill or a large decode batch is
 *   moe_rmsnorm -> (router) -> moe_dispatch_fused -> moe_expert_gemm_swiglu
 *   -> moe_expert_gemm -> moe_combine;
 * for a few tokens it is moe_rmsnorm -> (router) -> moe_layer_fused.  A shared
 * expert (or any dense layer) runs the two products with a NULL handle on the
 * 8-bit rows of moe_rmsnorm.
 *
 * The conventions of moe_dispatch.h hold: device pointers owned by the caller,
 * dense row-major arrays, no allocation, no synchronization, no state kept
 * between calls, argument errors returned before anything is enqueued, work
 * enqueued on `stream` and capturable in a HIP graph.  Results do not depend
 * on timing: no sum's order is left to the scheduling.
 *
 * Values that are not finite: a product with a NaN is NaN, and 8-bit rows keep
 * it (E4M3 NaN) beside the scale of the block's other values.  A block with an
 * infinite value has the scale +infinity and NaN in its place (FP8_F32), or
 * the scale 2^120 and +-448 (UE8M0, MXFP8); what is small against its scale is
 * 0.  Rows and tokens are independent: none shows in another's result.
 *
 * Weight formats, by cfg.quant (w has `n` output channels of `k` input
 * channels per expert):
 *   FP8_F32    w E4M3 [E, n, k], w_scale fp32 [E, ceil(n/128), k/128]
 *   FP8_UE8M0  w E4M3 [E, n, k], w_scale uint32 [E, ceil(n/128), ceil(k/512)]:
 *              byte b%4 of word b/4 = exponent byte (2^(byte-127)) of block b
 *   MXFP8      w E4M3 [E, n, k], w_scale uint8 [E, n, k/32] (E8M0)
 *   NONE       w bf16 [E, n, k], w_scale NULL (moe_layer_fused only)
 * Exponent byte 255 is NaN.  moe_layer_fused multiplies weights of UE8M0 and
 * MXFP8 as the bf16 values they stand for: what lies below bf16's range is lost
 * (bytes 0 to 2) or beyond it infinite (bytes from 247), the bytes between are
 * exact.
 */
#ifndef MOE_EXPERTS_H
#define MOE_EXPERTS_H

#include "moe_dispatch.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_LAYER_MAX_TOKENS 64 /* tokens one moe_layer_fused call takes */
#define MOE_NORM_MAX_HIDDEN 32768

/*
 * Residual add and root-mean-square norm of token rows:
 *   r   = residual != NULL ? bf16(x + residual) : x
 *   y   = r * (1 / sqrt(mean(r^2) + eps)) * weight         (fp32)
 *   residual_out = r, out = bf16(y),
 *   (out_q, out_scale) = y quantized as moe_dispatch quantizes (cfg.quant),
 *   from the fp32 y: one rounding to E4M3, not two.
 * The sum of squares is held in fp32: where it overflows (an r of 2^64 and
 * more) y is 0.
 *
 *   x             bf16 bits [num_tokens, H].
 *   residual      optional bf16 bits [num_tokens, H].
 *   weight        bf16 bits [H].
 *   eps           > 0 and finite.
 *   residual_out  bf16 bits [num_tokens, H]; required with residual (may be the
 *                 same array), NULL without.
 *   out           optional bf16 bits [num_tokens, H] (may be x's array).
 *   out_q         E4M3 [num_tokens, H] and
 *   out_scale     its scales in moe_dispatch's layout of out_scale with
 *                 num_tokens rows: both given or both NULL; NULL for quant NONE.
 * At least one of out and out_q is given.  cfg.hidden is H, at most
 * MOE_NORM_MAX_HIDDEN (larger: MOE_ERR_UNSUPPORTED).
 */
moe_status_t moe_rmsnorm(const moe_config_t *cfg, int32_t num_tokens, const uint16_t *x, const uint16_t *residual,
                         const uint16_t *weight, float eps, uint16_t *residual_out, uint16_t *out, void *out_q,
                         void *out_scale, void *stream);

/*
 * Expert products: for every row of expert e that holds a pair,
 *   y[row, j] = bf16( sum over blocks b of sa[row, b] * sw[e, j, b] *
 *                     sum over channels c of b of a[row, c] * w[e, j, c] )
 * blocks of 128 channels (32 for MXFP8).  Rows holding no pair are neither read
 * nor written.
 *
 * Precision: blocks are added in fp32.  Inside a block the 8-bit matrix
 * instruction adds the exact products of eight adjacent channels at a time (8 i
 * .. 8 i + 7) and drops from each what lies 13 binary places below the largest
 * of the eight: at most 7 * 2^-13 of that product per group of eight, scaled as
 * it is.  That lies below bf16's rounding unless loud channels cancel.  Few
 * rows share the sum among more waves, in another fixed order, so a row may
 * differ in its last bit between calls of different sizes.
 *
 *   n          output channels, a multiple of 8.
 *   k          input channels, a multiple of 128.  n and k are at most 2^22 and
 *              n * k / 32 < 2^31 (larger: MOE_ERR_UNSUPPORTED).
 *   a          E4M3 [rows, k] and a_scale its scales in moe_dispatch's layout of
 *              out_scale (k in the place of H): dispatched rows, or the rows of
 *              moe_expert_gemm_swiglu.
 *   handle     the handle of the dispatch that laid the rows out (recv_count and
 *              expert_offset are read): rows = moe_rows_capacity(cfg).  NULL: a
 *              dense layer -- cfg.num_experts must be 1 and the rows are the
 *              num_tokens rows of a.
 *   y          bf16 bits [rows, n].
 * cfg.quant is an FP8 format (NONE: MOE_ERR_UNSUPPORTED); cfg.hidden is not
 * read.  num_tokens is the batch of the dispatch: it sizes the launch, so the
 * handle must hold at most num_tokens * K pairs.
 */
moe_status_t moe_expert_gemm(const moe_config_t *cfg, int32_t num_tokens, int32_t n, int32_t k, const void *a,
                             const void *a_scale, const void *w, const void *w_scale, const moe_handle_t *handle,
                             uint16_t *y, void *stream);

/*
 * Gate and up products with SwiGLU: with g and u the products (not rounded to
 * bf16) of row `row` with output channels [0, inter) and [inter, 2*inter) of w13
 * [E, 2*inter, cfg.hidden],
 *   (h, h_scale)[row] = quantize( g / (1 + exp(-g)) * u )
 * as moe_dispatch quantizes (cfg.quant), inter in the place of H: the input of
 * moe_expert_gemm for the down product.  inter is a multiple of 128; a, handle,
 * num_tokens and the rows that are skipped as in moe_expert_gemm with
 * k = cfg.hidden.
 *
 * Precision: FP8_F32, whose stored scales show it, sums exact products in fp32;
 * UE8M0 and MXFP8 as moe_expert_gemm.  A row's result does not depend on the
 * rows beside it or on their number.
 */
moe_status_t moe_expert_gemm_swiglu(const moe_config_t *cfg, int32_t num_tokens, int32_t inter, const void *a,
                                    const void *a_scale, const void *w13, const void *w13_scale,
                                    const moe_handle_t *handle, void *h, void *h_scale, void *stream);

/* Bytes of device workspace moe_layer_fused needs for up to cfg.max_tokens
 * tokens (at most MOE_LAYER_MAX_TOKENS per call).  Returns 0 for a config or
 * inter that it refuses. */
size_t moe_layer_workspace_bytes(const moe_config_t *cfg, int32_t inter);

/*
 * A whole expert layer for a few tokens, in two kernels and without a dispatch:
 *   h[t,k]  = bf16( silu(W13[e] gate rows . x[t]) * (W13[e] up rows . x[t]) ),
 *   out[t]  = bf16( sum over k of topk_w[t,k] * W2[e] . h[t,k] ),  e = topk_idx[t,k]
 * with bf16 activations (no 8-bit rounding: a few tokens are bound by the
 * weights' bytes, not by the activations'), weights in cfg.quant's weight
 * format, and fp32 sums.  Pairs with an id outside [0, E) are skipped as in
 * moe_dispatch_layout (their weight is not read); a token without pairs gives
 * +0.  The same expert twice in one token counts twice.
 *
 *   inter      a multiple of 128, at most 2^27 (larger: MOE_ERR_UNSUPPORTED);
 *              cfg.hidden too, for every format.
 *   topk_idx   int32 [num_tokens, K]; topk_w fp32 [num_tokens, K].
 *   x          bf16 bits [num_tokens, H].
 *   w13        [E, 2*inter, H] (gate rows first), w2 [E, H, inter].
 *   workspace  >= moe_layer_workspace_bytes(cfg, inter) bytes, 16-byte aligned,
 *              clobbered: two calls that may overlap need one each.
 *   out        bf16 bits [num_tokens, H]; must not overlap x.
 * num_tokens > MOE_LAYER_MAX_TOKENS: MOE_ERR_UNSUPPORTED.  cfg's layout fields
 * are checked but not used.
 */
moe_status_t moe_layer_fused(const moe_config_t *cfg, int32_t num_tokens, int32_t inter, const int32_t *topk_idx,
                             const float *topk_w, const uint16_t *x, const void *w13, const void *w13_scale,
                             const void *w2, const void *w2_scale, void *workspace, size_t workspace_bytes,
                             uint16_t *out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H */
