// Internal declarations of the bf16 expert layer and its gradients
// (include/moe_train.h).
#pragma once

#include "moe_experts_internal.h"
#include "moe_train.h"

namespace moe {

// ---- products -------------------------------------------------------------------

enum TrainProduct { kLinear, kGated, kGradInput };

struct TrainGemmArgs {
    const uint16_t *rows;          // [rows, k] (kGradInput: [rows, n])
    const uint16_t *w;             // [E, n, k]; kGated: n = 2 * inter
    const int32_t *recv_count;     // [E]; NULL: one group of dense_rows rows
    const int32_t *expert_offset;  // [E + 1]; NULL with recv_count
    const uint16_t *bias;          // or NULL
    const uint16_t *residual;      // or NULL
    uint16_t *y;                   // [rows, n], kGated: [rows, n / 2], kGradInput: [rows, k]
    void *saved;                   // or NULL
    void *saved_scale;
    int32_t saved_quant, act;
    int32_t E, n, k, dense_rows;
    int64_t max_rows;              // rows that may hold pairs, all experts together (sizes the launch)
};
hipError_t launch_train_gemm(const TrainGemmArgs &a, TrainProduct product, hipStream_t stream);

struct GradWeightArgs {
    const uint16_t *dy;            // [rows, n]
    const void *a;                 // [rows, k] bf16 or E4M3
    const void *a_scale;
    const int32_t *recv_count, *expert_offset;
    void *dw;                      // [E, n, k] fp32 or bf16
    float *dbias;                  // or NULL
    float *partial;                // workspace: [E, splits, n, k], then [E, splits, n]
    int32_t a_quant, dw_bf16, accumulate, splits;
    int32_t E, n, k, dense_rows;
    int64_t max_rows;              // as above (chooses the tiles)
};
// Parts that an expert's rows are split into (1: no workspace).
int32_t grad_weight_splits(int64_t max_rows, int32_t E, int32_t n, int32_t k);
hipError_t launch_grad_weight(const GradWeightArgs &a, hipStream_t stream);

// ---- rows ------------------------------------------------------------------------

struct ActBackwardArgs {
    const uint16_t *dy;
    const void *saved;
    const void *saved_scale;
    const int32_t *row_to_pair;    // NULL: every row
    uint16_t *dsaved;
    uint16_t *y;                   // or NULL
    int32_t rows, n, act, quant;
};
hipError_t launch_activation_backward(const ActBackwardArgs &a, bool gated, hipStream_t stream);

struct CombineBackwardArgs {
    const uint16_t *dout;
    const uint16_t *y;             // or NULL
    const float *topk_w;
    const int32_t *pair_to_row;
    uint16_t *dy;
    float *dtopk_w;                // or NULL
    int32_t T, K, H;
};
hipError_t launch_combine_backward(const CombineBackwardArgs &a, hipStream_t stream);

}  // namespace moe
