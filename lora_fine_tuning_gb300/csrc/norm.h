// Launch plans of the norms around a block (norm.cuh, k_norm_fwd.cu, norm_bwd.cuh), filled by norm_api.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace lora {

constexpr int kNormMaxWidth = 16384;

// A vector of weights in bf16 or fp32, or none.
struct NormVec {
    const void* p;
    int32_t f32;
};

struct NormAct8 {
    uint8_t *codes, *scales;   // none where null
};

// What the forward and the backward have in common.
struct NormShape {
    int32_t rows, width;
    int32_t ragged;                     // some matrix has rows that do not start on 16 bytes or are not whole units of eight values
    int32_t vectors;                    // w, post and gate are whole vectors of eight values on 16-byte boundaries
    int32_t f32;                        // the stream is fp32
    NormVec w, post, gate, row_gate;
    float eps, offset, res, inv_width;
    int64_t codes_ld, scales_ld;
};

struct NormFwd {
    NormShape s;
    const void* h;
    const uint16_t* y;                  // may be null
    void* h_out;                        // null where y is
    uint16_t* x;                        // null where w is
    int64_t h_ld, y_ld, h_out_ld, x_ld;   // bytes
    NormAct8 x8, h8, y8;
    int32_t stages;                     // of a row group's ring in shared memory, and their bytes (the launch sets them)
    uint32_t stage_bytes, at_y;
};

struct NormBwd {
    NormShape s;
    const uint16_t* dx;                 // null where w is
    const void* dh;                     // may be null: zero
    const void* h;                      // the forward's h_out; null where h8 has it
    const uint16_t* y;                  // may be null (or y8)
    void* dh_out;
    uint16_t* dy;                       // may be null
    int64_t dx_ld, dh_ld, h_ld, y_ld, dh_out_ld, dy_ld;   // bytes
    NormAct8 h8, y8;
    float* part;                        // sums over each group's rows: groups x 2 x width; null: no weights' gradients
    float *dw, *dpost, *dgate, *drow;   // each may be null
    // set by the launch
    int32_t groups, stages;
    uint32_t stage_bytes, at_dx, at_h, at_dh, at_y;
};

// The most groups of rows that the backward sums over: the partial sums' first extent.
int norm_bwd_groups(int rows, int width, int sms);

cudaError_t launch_norm_fwd(const NormFwd& p, int sms, cudaStream_t stream);
cudaError_t launch_norm_bwd(NormBwd& p, int sms, cudaStream_t stream);        // without the weights' gradients
cudaError_t launch_norm_bwd_sums(NormBwd& p, int sms, cudaStream_t stream);   // with their sums over each CTA's rows
cudaError_t launch_norm_bwd8(NormBwd& p, int sms, cudaStream_t stream);       // the same where h or y is in 8 bits
cudaError_t launch_norm_bwd8_sums(NormBwd& p, int sms, cudaStream_t stream);
cudaError_t launch_norm_sums(const NormBwd& p, cudaStream_t stream);

}  // namespace lora
