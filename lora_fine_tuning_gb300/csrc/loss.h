// Launch plans of the losses on logits (k_loss.cu), filled by loss_api.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "plan.h"

namespace lora {

constexpr int kLossMaxPairs = 1024;

struct LossLogits {
    const void* z;         // rows x vocab, row stride ld elements
    void* dz;              // may be null (no gradient) or z itself
    int64_t rows, ld, dz_ld;
    int32_t vocab;
    int32_t f32;           // fp32 (else bf16)
    const int64_t* labels; // a row whose label is outside [0, vocab) does not count
    float* logp;           // rows: log p of the label, 0 where there is none
};

// Statistics of a row kept between the passes: its maximum and 1 / sum exp(z - maximum).
struct LossRow {
    float top, inv;
};

struct PrefParams {
    LossLogits in;
    const float* ref;      // rows, may be null
    LossRow* row;          // workspace, rows
    float* coef;           // workspace, rows: d loss / d logp
    float* loss;           // 1
    float* margin;         // pairs
    float* pair_loss;      // workspace, pairs
    uint32_t* ticket;      // workspace, zero between calls
    int32_t n_pairs;
    float beta, smoothing, scale;
    DevCtl ctl;
};

struct PrefPair {
    int32_t chosen, rejected, chosen_rows, rejected_rows;
};
template <int N>
struct PrefPairs {
    PrefPair p[N];
};
constexpr int kFewPairs = 64;

// For long rows: with few and short pairs the pass over the logits also forms the pairs' losses (`fused`): a warp a pair.
constexpr int kFusedPairs = 16;
constexpr int kFusedPairRows = 128;
struct PrefLong : PrefParams {
    int32_t fused;
    PrefPairs<kFusedPairs> pairs;
};

struct PolicyParams {
    LossLogits in;
    const float *old_logp, *adv, *ref;   // rows; ref may be null
    float* row_loss;       // workspace, rows
    uint32_t* ticket;      // workspace, zero between calls
    float* loss;           // 1
    float lo, hi;          // 1 - clip_low, 1 + clip_high
    float kl, scale;
    DevCtl ctl;
};

// *paired: the kernel also formed the pairs' losses (launch_loss_pairs otherwise).
cudaError_t launch_loss_stats(const PrefParams& p, const PrefPairs<kLossMaxPairs>& pairs, int sms, bool* paired, cudaStream_t stream);
cudaError_t launch_loss_pairs(const PrefParams& p, const PrefPairs<kLossMaxPairs>& pairs, cudaStream_t stream);
cudaError_t launch_loss_grad(const PrefParams& p, cudaStream_t stream);
// *summed: the kernel also wrote the loss (launch_loss_sum otherwise).
cudaError_t launch_policy_rows(const PolicyParams& p, int sms, bool* summed, cudaStream_t stream);
cudaError_t launch_loss_sum(const float* x, int64_t n, float scale, float* out, cudaStream_t stream);

}  // namespace lora
