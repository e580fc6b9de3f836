// Internal declarations of the expert-layer operators (include/moe_experts.h).
#pragma once

#include "moe_experts.h"
#include "moe_internal.h"

namespace moe {

// Host checks shared with the dispatch entry points (moe_abi.hip).
bool aligned(const void *p, size_t a);
moe_status_t check_config(const moe_config_t *cfg);
moe_status_t check_handle(const moe_handle_t *h);
moe_status_t check_tokens(const moe_config_t &c, int32_t num_tokens);

// ---- residual add + norm ------------------------------------------------------

struct NormArgs {
    const uint16_t *x;
    const uint16_t *residual;      // or NULL
    const uint16_t *weight;
    uint16_t *residual_out;        // with residual only
    uint16_t *out;                 // or NULL
    uint8_t *out_q;                // or NULL
    void *out_scale;
    float eps;
    int32_t T, H;
};
hipError_t launch_rmsnorm(const NormArgs &a, int32_t quant, hipStream_t stream);

// ---- grouped products -----------------------------------------------------------

// Channels of a product: the 256 rows of a tile, read or written, stay within
// 2 GiB of 32-bit offsets.
constexpr int32_t kMaxGemmK = 1 << 22, kMaxGemmN = 1 << 22;

struct ExpertGemmArgs {
    const uint8_t *a;              // [rows, k] E4M3
    const void *a_scale;
    const uint8_t *w;              // [E, n, k] E4M3
    const void *w_scale;
    const int32_t *recv_count;     // [E]; NULL: one group of dense_rows rows
    const int32_t *expert_offset;  // [E + 1]; NULL with recv_count
    uint16_t *y;                   // [rows, n] bf16 (plain product)
    uint8_t *h;                    // [rows, inter] E4M3 (SwiGLU; n = 2 * inter)
    void *h_scale;
    int32_t E, n, k, dense_rows;
    int64_t max_rows;              // rows that may hold pairs, all experts together (sizes the launch)
};
hipError_t launch_expert_gemm(const ExpertGemmArgs &a, int32_t quant, bool swiglu, hipStream_t stream);

// ---- few-token layer --------------------------------------------------------------

// Channels of the layer, inner or outer: its grids' threads (16 or 32 channels per
// block of 256 or 512) are counted in 32 bits and would wrap without an error.
constexpr int32_t kMaxLayerChannels = 1 << 27;

struct LayerArgs {
    const int32_t *topk_idx;
    const float *topk_w;
    const uint16_t *x;
    const uint8_t *w13;
    const void *w13_scale;
    const uint8_t *w2;
    const void *w2_scale;
    uint64_t *masks;               // workspace: tokens of each expert slot [min(T * K, E)]
    uint16_t *h;                   // workspace: bf16 [T * K, inter]
    uint16_t *out;
    int32_t T, K, E, H, I;
};
hipError_t launch_layer(const LayerArgs &a, int32_t quant, hipStream_t stream);

}  // namespace moe
