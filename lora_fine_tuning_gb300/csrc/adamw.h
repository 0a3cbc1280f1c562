// Launch plan of the AdamW step (k_adamw.cu), filled by adamw_api.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace lora {

constexpr int kAdamBlock = 256;        // values that share a scale in the 8-bit states
constexpr int kAdamChunk8 = 4096;      // values of one CTA: 8-bit states
constexpr int kAdamChunk32 = 2048;     // fp32 states
constexpr int kAdamTensors = 384;      // tensors of one launch (the table is a kernel parameter)

enum : uint32_t { kAdamParamF32 = 1, kAdamGradF32 = 2 };

struct AdamTensor {
    void* param;
    const void* grad;
    void *m, *v;
    float *m_scale, *v_scale;   // 8-bit states only
    float* master;              // may be null
    int64_t n;
    uint32_t flags;
};

struct AdamStep {
    float b1, b1c, b2, b2c;     // beta and 1 - beta
    float keep;                 // 1 - lr * weight_decay
    float rate;                 // -lr / (1 - beta1^t)
    float inv_c2;               // 1 / sqrt(1 - beta2^t)
    float eps;
    float one;                  // 1 (k_adamw.cu)
    const float* grad_scale;    // may be null
    int32_t n;
};

template <int N>
struct AdamTensors {
    AdamTensor t[N];
    int32_t chunk0[N];          // first chunk of each tensor in the launch
};
constexpr int kAdamFew = 32;

// Only the first p.n entries of the table are read.
cudaError_t launch_adamw(const AdamStep& p, const AdamTensors<kAdamTensors>& t, bool bits8, int chunks,
                         cudaStream_t stream);

}  // namespace lora
