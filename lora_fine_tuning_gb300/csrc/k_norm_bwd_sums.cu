// The backward of the norms around a block with the weights' gradients.
#include "norm_bwd.cuh"

namespace lora {

namespace {

// The CTAs' sums added in a fixed order: a warp's lanes have 32 columns, and each of the CTA's warps adds every kSumWarps-th group.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32) norm_sums_kernel(const __grid_constant__ NormBwd p) {
    __shared__ float part[2][kSumWarps][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, width = p.s.width;
    float a = 0.f, b = 0.f;
    if (c < width) {
        const float* at = p.part + c;
        const int64_t one = 2 * static_cast<int64_t>(width);
#pragma unroll 8
        for (int g = warp; g < p.groups; g += kSumWarps) {
            a += __ldcg(at + g * one);
            b += __ldcg(at + g * one + width);
        }
    }
    part[0][warp][lane] = a;
    part[1][warp][lane] = b;
    __syncthreads();
    if (warp != 0 || c >= width) return;
#pragma unroll
    for (int i = 1; i < kSumWarps; ++i) {
        a += part[0][i][lane];
        b += part[1][i][lane];
    }
    if (p.dw) p.dw[c] = a;
    const float w = p.s.post.p ? one_weight(p.s.post, c) + p.s.offset : 1.f;
    if (p.dgate) p.dgate[c] = p.s.res * w * b;
    if (p.dpost) p.dpost[c] = p.s.res * (p.s.gate.p ? one_weight(p.s.gate, c) : 1.f) * b;
}

}  // namespace

// The most groups of rows that any form of the backward has: its CTAs.
int norm_bwd_groups(int rows, int width, int sms) {
    const auto groups = [&](bool ragged) {
        return by_width(width, ragged, [&](auto t, auto, auto) {
            constexpr int T = decltype(t)::value, R = rows_of(T);
            return std::min((rows + R - 1) / R, sms * per_sm(T));
        });
    };
    return std::max(groups(false), groups(true));
}

cudaError_t launch_norm_bwd_sums(NormBwd& p, int sms, cudaStream_t stream) {
    return launch_norm_bwd_form<true, false>(p, sms, stream);
}

cudaError_t launch_norm_sums(const NormBwd& p, cudaStream_t stream) {
    return launch_pdl(norm_sums_kernel, dim3((p.s.width + 31) / 32), dim3(kSumWarps * 32), 0, stream, p);
}

}  // namespace lora
