// C ABI of the bf16 expert layer and its gradients (include/moe_train.h):
// argument checks and launches.  Every argument error is found here, before
// anything is enqueued.
#include "moe_train_internal.h"

namespace moe {

namespace {

moe_status_t from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

bool pointer(const void *p, size_t align) { return p != nullptr && aligned(p, align); }

bool known_quant(int32_t q) { return q >= MOE_QUANT_NONE && q <= MOE_QUANT_MXFP8; }

bool known_act(int32_t act) { return act >= MOE_ACT_NONE && act <= MOE_ACT_RELU; }

// Config, handle (NULL: one dense group) and tokens.
moe_status_t check_rows(const moe_config_t *cfg, int32_t num_tokens, const moe_handle_t *handle)
{
    moe_status_t st = check_config(cfg);
    if (st != MOE_OK)
        return st;
    if (handle != nullptr && (st = check_handle(handle)) != MOE_OK)
        return st;
    if ((st = check_tokens(*cfg, num_tokens)) != MOE_OK)
        return st;
    return handle == nullptr && cfg->num_experts != 1 ? MOE_ERR_INVALID_ARG : MOE_OK;
}

moe_status_t check_channels(int32_t c)
{
    if (c < 8 || c % 8 != 0)
        return MOE_ERR_INVALID_ARG;
    return c > MOE_TRAIN_MAX_CHANNELS ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Rows and scales of a format; `block` channels hold whole blocks of scales.
bool formatted(int32_t quant, const void *rows, const void *scale, int32_t block)
{
    if (!pointer(rows, 16))
        return false;
    if (quant == MOE_QUANT_NONE)
        return scale == nullptr;
    return pointer(scale, 4) && block % kQuantGroup == 0;
}

// Rows that may hold pairs, all experts together.
int64_t most_rows(const moe_config_t &c, int32_t num_tokens, const moe_handle_t *handle)
{
    if (handle == nullptr)
        return num_tokens;
    const int64_t pairs = (int64_t)num_tokens * c.num_topk, slab = (int64_t)c.num_experts * c.capacity;
    return c.layout == MOE_LAYOUT_MASKED && slab < pairs ? slab : pairs;
}

TrainGemmArgs product_args(const moe_config_t &c, int32_t num_tokens, int32_t n, int32_t k, const uint16_t *rows,
                           const uint16_t *w, const moe_handle_t *handle, uint16_t *y)
{
    TrainGemmArgs p = {};
    p.rows = rows;
    p.w = w;
    p.recv_count = handle != nullptr ? handle->recv_count : nullptr;
    p.expert_offset = handle != nullptr ? handle->expert_offset : nullptr;
    p.y = y;
    p.saved_quant = MOE_QUANT_NONE;
    p.act = MOE_ACT_NONE;
    p.E = c.num_experts;
    p.n = n;
    p.k = k;
    p.dense_rows = num_tokens;
    p.max_rows = most_rows(c, num_tokens, handle);
    return p;
}

// Saved rows of a forward product; `block`: channels that hold whole blocks.
moe_status_t check_saved(const void *saved, const void *saved_scale, int32_t saved_quant, int32_t block)
{
    if (!known_quant(saved_quant))
        return MOE_ERR_INVALID_ARG;
    if (saved == nullptr)
        return saved_scale == nullptr ? MOE_OK : MOE_ERR_INVALID_ARG;
    return formatted(saved_quant, saved, saved_scale, block) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

size_t grad_weight_bytes(const moe_config_t &c, int64_t max_rows, int32_t n, int32_t k)
{
    const int32_t splits = grad_weight_splits(max_rows, c.num_experts, n, k);
    return splits == 1 ? 0 : (size_t)splits * c.num_experts * ((size_t)n * k + n) * sizeof(float);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_ffn_gated(const moe_config_t *cfg, int32_t num_tokens, int32_t inter, int32_t act,
                           const uint16_t *a, const uint16_t *w13, const moe_handle_t *handle, uint16_t *h,
                           void *saved, void *saved_scale, int32_t saved_quant, void *stream)
{
    moe_status_t st = check_rows(cfg, num_tokens, handle);
    if (st != MOE_OK)
        return st;
    if (!known_act(act))
        return MOE_ERR_INVALID_ARG;
    if (inter > MOE_TRAIN_MAX_CHANNELS / 2)
        return MOE_ERR_UNSUPPORTED;
    if ((st = check_channels(inter)) != MOE_OK || (st = check_channels(cfg->hidden)) != MOE_OK)
        return st;
    if ((st = check_saved(saved, saved_scale, saved_quant, inter)) != MOE_OK || num_tokens == 0)
        return st;
    if (!pointer(a, 16) || !pointer(w13, 16) || !pointer(h, 16))
        return MOE_ERR_INVALID_ARG;
    TrainGemmArgs p = product_args(*cfg, num_tokens, 2 * inter, cfg->hidden, a, w13, handle, h);
    p.act = act;
    p.saved = saved;
    p.saved_scale = saved_scale;
    p.saved_quant = saved_quant;
    return from_hip(launch_train_gemm(p, kGated, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_expert_linear(const moe_config_t *cfg, int32_t num_tokens, int32_t n, int32_t k, int32_t act,
                               const uint16_t *a, const uint16_t *w, const uint16_t *bias, const uint16_t *residual,
                               const moe_handle_t *handle, uint16_t *y, void *saved, void *saved_scale,
                               int32_t saved_quant, void *stream)
{
    moe_status_t st = check_rows(cfg, num_tokens, handle);
    if (st != MOE_OK)
        return st;
    if (!known_act(act))
        return MOE_ERR_INVALID_ARG;
    if ((st = check_channels(n)) != MOE_OK || (st = check_channels(k)) != MOE_OK)
        return st;
    if ((st = check_saved(saved, saved_scale, saved_quant, n)) != MOE_OK || num_tokens == 0)
        return st;
    if (!pointer(a, 16) || !pointer(w, 16) || !pointer(y, 16) || !aligned(bias, 16) || !aligned(residual, 16))
        return MOE_ERR_INVALID_ARG;
    TrainGemmArgs p = product_args(*cfg, num_tokens, n, k, a, w, handle, y);
    p.act = act;
    p.bias = bias;
    p.residual = residual;
    p.saved = saved;
    p.saved_scale = saved_scale;
    p.saved_quant = saved_quant;
    return from_hip(launch_train_gemm(p, kLinear, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_activation_backward(const moe_config_t *cfg, int32_t num_tokens, int32_t n, int32_t act,
                                     int32_t gated, const uint16_t *dy, const void *saved, const void *saved_scale,
                                     int32_t saved_quant, const moe_handle_t *handle, uint16_t *dsaved, uint16_t *y,
                                     void *stream)
{
    moe_status_t st = check_rows(cfg, num_tokens, handle);
    if (st != MOE_OK)
        return st;
    if (!known_act(act) || !known_quant(saved_quant) || (gated != 0 && gated != 1))
        return MOE_ERR_INVALID_ARG;
    if (gated && n > MOE_TRAIN_MAX_CHANNELS / 2)
        return MOE_ERR_UNSUPPORTED;
    if ((st = check_channels(n)) != MOE_OK || num_tokens == 0)
        return st;
    if (!formatted(saved_quant, saved, saved_scale, n) || !pointer(dy, 16) || !pointer(dsaved, 16) || !aligned(y, 16))
        return MOE_ERR_INVALID_ARG;
    ActBackwardArgs a = {};
    a.dy = dy;
    a.saved = saved;
    a.saved_scale = saved_scale;
    a.row_to_pair = handle != nullptr ? handle->row_to_pair : nullptr;
    a.dsaved = dsaved;
    a.y = y;
    a.rows = handle != nullptr ? (int32_t)moe_rows_capacity(cfg) : num_tokens;
    a.n = n;
    a.act = act;
    a.quant = saved_quant;
    return from_hip(launch_activation_backward(a, gated != 0, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_expert_grad_input(const moe_config_t *cfg, int32_t num_tokens, int32_t n, int32_t k,
                                   const uint16_t *dy, const uint16_t *w, const moe_handle_t *handle, uint16_t *da,
                                   void *stream)
{
    moe_status_t st = check_rows(cfg, num_tokens, handle);
    if (st != MOE_OK)
        return st;
    if ((st = check_channels(n)) != MOE_OK || (st = check_channels(k)) != MOE_OK || num_tokens == 0)
        return st;
    if (!pointer(dy, 16) || !pointer(w, 16) || !pointer(da, 16))
        return MOE_ERR_INVALID_ARG;
    const TrainGemmArgs p = product_args(*cfg, num_tokens, n, k, dy, w, handle, da);
    return from_hip(launch_train_gemm(p, kGradInput, static_cast<hipStream_t>(stream)));
}

size_t moe_grad_weight_workspace_bytes(const moe_config_t *cfg, int32_t num_tokens, int32_t n, int32_t k)
{
    if (check_config(cfg) != MOE_OK || check_tokens(*cfg, num_tokens) != MOE_OK || check_channels(n) != MOE_OK ||
        check_channels(k) != MOE_OK)
        return 0;
    // with a handle or without: the larger of both
    const int64_t rows = (int64_t)num_tokens * cfg->num_topk;
    return grad_weight_bytes(*cfg, rows, n, k);
}

moe_status_t moe_expert_grad_weight(const moe_config_t *cfg, int32_t num_tokens, int32_t n, int32_t k,
                                    const uint16_t *dy, const void *a, const void *a_scale, int32_t a_quant,
                                    const moe_handle_t *handle, void *dw, int32_t dw_bf16, float *dbias,
                                    int32_t accumulate, void *workspace, size_t workspace_bytes, void *stream)
{
    moe_status_t st = check_rows(cfg, num_tokens, handle);
    if (st != MOE_OK)
        return st;
    if (!known_quant(a_quant) || (dw_bf16 != 0 && dw_bf16 != 1) || (accumulate != 0 && accumulate != 1) ||
        (dw_bf16 && accumulate))
        return MOE_ERR_INVALID_ARG;
    if ((st = check_channels(n)) != MOE_OK || (st = check_channels(k)) != MOE_OK)
        return st;
    if (a_quant != MOE_QUANT_NONE && k % kQuantGroup != 0)
        return MOE_ERR_INVALID_ARG;
    if (num_tokens > 0 && (!formatted(a_quant, a, a_scale, k) || !pointer(dy, 16)))
        return MOE_ERR_INVALID_ARG;
    if (!pointer(dw, 16) || !aligned(dbias, 4))
        return MOE_ERR_INVALID_ARG;
    const int64_t rows = most_rows(*cfg, num_tokens, handle);
    const size_t need = grad_weight_bytes(*cfg, rows, n, k);
    if (need > 0 && !pointer(workspace, 16))
        return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < need)
        return MOE_ERR_CAPACITY;
    GradWeightArgs p = {};
    p.dy = dy;
    p.a = a;
    p.a_scale = a_scale;
    // no tokens: no expert has rows, whatever the handle holds
    p.recv_count = handle != nullptr && num_tokens > 0 ? handle->recv_count : nullptr;
    p.expert_offset = handle != nullptr && num_tokens > 0 ? handle->expert_offset : nullptr;
    p.dw = dw;
    p.dbias = dbias;
    p.partial = static_cast<float *>(workspace);
    p.a_quant = a_quant;
    p.dw_bf16 = dw_bf16;
    p.accumulate = accumulate;
    p.splits = grad_weight_splits(rows, cfg->num_experts, n, k);
    p.E = cfg->num_experts;
    p.n = n;
    p.k = k;
    p.dense_rows = num_tokens;
    p.max_rows = rows;
    return from_hip(launch_grad_weight(p, static_cast<hipStream_t>(stream)));
}

moe_status_t moe_combine_backward(const moe_config_t *cfg, int32_t num_tokens, const uint16_t *dout,
                                  const uint16_t *y, const float *topk_w, const moe_handle_t *handle, uint16_t *dy,
                                  float *dtopk_w, void *stream)
{
    moe_status_t st = check_config(cfg);
    if (st != MOE_OK)
        return st;
    if ((st = check_handle(handle)) != MOE_OK)
        return st;
    if ((st = check_tokens(*cfg, num_tokens)) != MOE_OK || (st = check_channels(cfg->hidden)) != MOE_OK ||
        num_tokens == 0)
        return st;
    if (!pointer(dout, 16) || !pointer(topk_w, 4) || !pointer(dy, 16) || !aligned(y, 16) || !aligned(dtopk_w, 4) ||
        (y == nullptr) != (dtopk_w == nullptr))
        return MOE_ERR_INVALID_ARG;
    CombineBackwardArgs a = {};
    a.dout = dout;
    a.y = y;
    a.topk_w = topk_w;
    a.pair_to_row = handle->pair_to_row;
    a.dy = dy;
    a.dtopk_w = dtopk_w;
    a.T = num_tokens;
    a.K = cfg->num_topk;
    a.H = cfg->hidden;
    return from_hip(launch_combine_backward(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
