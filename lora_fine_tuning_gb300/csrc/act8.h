// Launch plans of the activations in 8 bits (k_act8.cu), filled by act8_api.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace lora {

// Codes lie in rows of whole blocks, scales in rows of whole words (four blocks, one word for 128 values).
__host__ __device__ inline int64_t act8_codes_ld(int64_t width) { return (width + 31) / 32 * 32; }
__host__ __device__ inline int64_t act8_scales_ld(int64_t width) { return (width + 127) / 128 * 4; }

struct Act8Params {
    uint16_t* x;           // rows x width, row stride ld elements (store: read only)
    uint8_t *codes, *scales;
    int64_t ld;
    int32_t width;
    uint32_t per_row;      // units of eight codes in a row of codes
    uint32_t units;        // rows * per_row
    int32_t vector;        // whole units of x are 16-byte aligned
    uint32_t magic, shift; // u / per_row = high word of (u magic) >> shift, for u below 2^31
};

cudaError_t launch_act8_store(const Act8Params& p, cudaStream_t stream);
cudaError_t launch_act8_load(const Act8Params& p, cudaStream_t stream);

}  // namespace lora
