// C ABI of the expert-layer operators (include/moe_experts.h): argument checks
// and launches.  Every argument error is found here, before anything is
// enqueued.
#include <limits.h>
#include <math.h>

#include "moe_experts_internal.h"

namespace moe {

namespace {

moe_status_t from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

bool pointer(const void *p, size_t align) { return p != nullptr && aligned(p, align); }

// Stored scales start where their words (or fp32 values) can be read whole.
bool weight(const moe_config_t &c, const void *w, const void *w_scale)
{
    if (!pointer(w, 16))
        return false;
    return c.quant == MOE_QUANT_NONE ? w_scale == nullptr : pointer(w_scale, 4);
}

// Checks shared by the two products; fills everything but the outputs.
moe_status_t prepare_gemm(const moe_config_t *cfg, int32_t num_tokens, int32_t n, int32_t k, const void *a,
                          const void *a_scale, const void *w, const void *w_scale, const moe_handle_t *handle,
                          const void *out, size_t out_align, ExpertGemmArgs &p)
{
    moe_status_t st = check_config(cfg);
    if (st != MOE_OK)
        return st;
    if (handle != nullptr && (st = check_handle(handle)) != MOE_OK)
        return st;
    if ((st = check_tokens(*cfg, num_tokens)) != MOE_OK)
        return st;
    if (cfg->quant == MOE_QUANT_NONE)
        return MOE_ERR_UNSUPPORTED;
    if (n < 8 || n % 8 != 0 || k < kQuantGroup || k % kQuantGroup != 0)
        return MOE_ERR_INVALID_ARG;
    // a tile's rows and an expert's weight scales are addressed with 32-bit offsets
    if (n > kMaxGemmN || k > kMaxGemmK || (int64_t)n * (k / 32) > INT32_MAX)
        return MOE_ERR_UNSUPPORTED;
    if (handle == nullptr && cfg->num_experts != 1)
        return MOE_ERR_INVALID_ARG;
    if (num_tokens > 0 && (!pointer(a, 16) || !pointer(a_scale, 4) || !weight(*cfg, w, w_scale) ||
                           !pointer(out, out_align)))
        return MOE_ERR_INVALID_ARG;
    p.a = static_cast<const uint8_t *>(a);
    p.a_scale = a_scale;
    p.w = static_cast<const uint8_t *>(w);
    p.w_scale = w_scale;
    p.recv_count = handle != nullptr ? handle->recv_count : nullptr;
    p.expert_offset = handle != nullptr ? handle->expert_offset : nullptr;
    p.y = nullptr;
    p.h = nullptr;
    p.h_scale = nullptr;
    p.E = cfg->num_experts;
    p.n = n;
    p.k = k;
    p.dense_rows = num_tokens;
    p.max_rows = num_tokens;
    if (handle != nullptr) {
        p.max_rows = (int64_t)num_tokens * cfg->num_topk;
        if (cfg->layout == MOE_LAYOUT_MASKED) {
            const int64_t slab = (int64_t)cfg->num_experts * cfg->capacity;
            p.max_rows = slab < p.max_rows ? slab : p.max_rows;
        }
    }
    return MOE_OK;
}

moe_status_t check_layer(const moe_config_t *cfg, int32_t inter)
{
    const moe_status_t st = check_config(cfg);
    if (st != MOE_OK)
        return st;
    if (inter < kQuantGroup || inter % kQuantGroup != 0 || cfg->hidden % kQuantGroup != 0)
        return MOE_ERR_INVALID_ARG;
    if (inter > kMaxLayerChannels || cfg->hidden > kMaxLayerChannels)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// Workspace of a call: the experts' token masks (room for every pair, in whole
// 16 bytes), then h.
size_t layer_mask_bytes(const moe_config_t &c, int32_t tokens)
{
    return ((size_t)tokens * c.num_topk * sizeof(uint64_t) + 15) / 16 * 16;
}

size_t layer_bytes(const moe_config_t &c, int32_t tokens, int32_t inter)
{
    const int32_t t = tokens < MOE_LAYER_MAX_TOKENS ? tokens : MOE_LAYER_MAX_TOKENS;
    return layer_mask_bytes(c, t) + (size_t)t * c.num_topk * inter * sizeof(uint16_t);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_rmsnorm(const moe_config_t *cfg, int32_t num_tokens, const uint16_t *x, const uint16_t *residual,
                         const uint16_t *weight, float eps, uint16_t *residual_out, uint16_t *out, void *out_q,
                         void *out_scale, void *stream)
{
    moe_status_t st = check_config(cfg);
    if (st != MOE_OK)
        return st;
    if ((st = check_tokens(*cfg, num_tokens)) != MOE_OK)
        return st;
    if (!(eps > 0.0f) || !isfinite(eps))
        return MOE_ERR_INVALID_ARG;
    if ((residual == nullptr) != (residual_out == nullptr) || (out_q == nullptr) != (out_scale == nullptr))
        return MOE_ERR_INVALID_ARG;
    if (cfg->quant == MOE_QUANT_NONE && out_q != nullptr)
        return MOE_ERR_INVALID_ARG;
    if (cfg->hidden > MOE_NORM_MAX_HIDDEN)
        return MOE_ERR_UNSUPPORTED;
    if (num_tokens == 0)
        return MOE_OK;
    if (!pointer(x, 16) || !pointer(weight, 16) || (out == nullptr && out_q == nullptr))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(residual, 16) || !aligned(residual_out, 16) || !aligned(out, 16) || !aligned(out_q, 16) ||
        !aligned(out_scale, 4))
        return MOE_ERR_INVALID_ARG;
    NormArgs a;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.residual_out = residual_out;
    a.out = out;
    a.out_q = static_cast<uint8_t *>(out_q);
    a.out_scale = out_scale;
    a.eps = eps;
    a.T = num_tokens;
    a.H = cfg->hidden;
    return from_hip(launch_rmsnorm(a, cfg->quant, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_expert_gemm(const moe_config_t *cfg, int32_t num_tokens, int32_t n, int32_t k, const void *a,
                             const void *a_scale, const void *w, const void *w_scale, const moe_handle_t *handle,
                             uint16_t *y, void *stream)
{
    ExpertGemmArgs p;
    const moe_status_t st = prepare_gemm(cfg, num_tokens, n, k, a, a_scale, w, w_scale, handle, y, 16, p);
    if (st != MOE_OK || num_tokens == 0)
        return st;
    p.y = y;
    return from_hip(launch_expert_gemm(p, cfg->quant, false, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_expert_gemm_swiglu(const moe_config_t *cfg, int32_t num_tokens, int32_t inter, const void *a,
                                    const void *a_scale, const void *w13, const void *w13_scale,
                                    const moe_handle_t *handle, void *h, void *h_scale, void *stream)
{
    if (cfg == nullptr || inter < kQuantGroup || inter % kQuantGroup != 0 || inter > INT32_MAX / 2)
        return MOE_ERR_INVALID_ARG;
    ExpertGemmArgs p;
    const moe_status_t st =
        prepare_gemm(cfg, num_tokens, 2 * inter, cfg->hidden, a, a_scale, w13, w13_scale, handle, h, 16, p);
    if (st != MOE_OK || num_tokens == 0)
        return st;
    if (!pointer(h_scale, 4))
        return MOE_ERR_INVALID_ARG;
    p.h = static_cast<uint8_t *>(h);
    p.h_scale = h_scale;
    return from_hip(launch_expert_gemm(p, cfg->quant, true, static_cast<hipStream_t>(stream)));
}

size_t moe_layer_workspace_bytes(const moe_config_t *cfg, int32_t inter)
{
    if (check_layer(cfg, inter) != MOE_OK)
        return 0;
    return layer_bytes(*cfg, cfg->max_tokens, inter);
}

moe_status_t moe_layer_fused(const moe_config_t *cfg, int32_t num_tokens, int32_t inter, const int32_t *topk_idx,
                             const float *topk_w, const uint16_t *x, const void *w13, const void *w13_scale,
                             const void *w2, const void *w2_scale, void *workspace, size_t workspace_bytes,
                             uint16_t *out, void *stream)
{
    moe_status_t st = check_layer(cfg, inter);
    if (st != MOE_OK)
        return st;
    if ((st = check_tokens(*cfg, num_tokens)) != MOE_OK)
        return st;
    if (num_tokens > MOE_LAYER_MAX_TOKENS)
        return MOE_ERR_UNSUPPORTED;
    if (num_tokens == 0)
        return MOE_OK;
    if (!pointer(topk_idx, 4) || !pointer(topk_w, 4) || !pointer(x, 16) || !weight(*cfg, w13, w13_scale) ||
        !weight(*cfg, w2, w2_scale) || !pointer(workspace, 16) || !pointer(out, 16))
        return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < layer_bytes(*cfg, num_tokens, inter))
        return MOE_ERR_CAPACITY;
    LayerArgs a;
    a.topk_idx = topk_idx;
    a.topk_w = topk_w;
    a.x = x;
    a.w13 = static_cast<const uint8_t *>(w13);
    a.w13_scale = w13_scale;
    a.w2 = static_cast<const uint8_t *>(w2);
    a.w2_scale = w2_scale;
    a.masks = static_cast<uint64_t *>(workspace);
    a.h = reinterpret_cast<uint16_t *>(static_cast<char *>(workspace) + layer_mask_bytes(*cfg, num_tokens));
    a.out = out;
    a.T = num_tokens;
    a.K = cfg->num_topk;
    a.E = cfg->num_experts;
    a.H = cfg->hidden;
    a.I = inter;
    return from_hip(launch_layer(a, cfg->quant, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
