// Activations into 8 bits and back (act8.cuh has the format).
//
// Bound by memory: 2 + 1.03 bytes a value in either direction.  The matrix is cut into units of eight values (16 bytes of
// bf16, 8 of codes), a lane a unit and four lanes a block, so a block's largest value takes two shuffles.  A CTA has
// kUnits consecutive units a thread, its loads all under way before the first is used.
#include "act8.cuh"
#include "act8.h"
#include "kernels.h"

namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;

// Eight values of a row from column c on; those past the row's end are zero.
template <bool kVec>
__device__ __forceinline__ uint4 load_unit(const uint16_t* row, int c, int width) {
    if (kVec && c + 8 <= width) return __ldcs(reinterpret_cast<const uint4*>(row + c));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < width) w[i / 2] |= static_cast<uint32_t>(row[c + i]) << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool kVec>
__device__ __forceinline__ void store_unit(uint16_t* row, int c, int width, uint4 x) {
    if (kVec && c + 8 <= width) {
        *reinterpret_cast<uint4*>(row + c) = x;
        return;
    }
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < width) row[c + i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
}

template <bool kVec>
__global__ void __launch_bounds__(kThreads) act8_store_kernel(const Act8Params p) {
    pdl_wait();
    pdl_trigger();
    const uint32_t u0 = blockIdx.x * (kThreads * kUnits) + threadIdx.x;
    uint4 x[kUnits];
    uint32_t row[kUnits], at[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t u = u0 + i * kThreads;
        row[i] = u / p.per_row;
        at[i] = u - row[i] * p.per_row;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (u < p.units) x[i] = load_unit<kVec>(p.x + row[i] * p.ld, static_cast<int>(at[i]) * 8, p.width);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t u = u0 + i * kThreads;
        uint32_t e;
        const uint2 c = act8_encode8(x[i], e);
        if (u >= p.units) continue;
        reinterpret_cast<uint2*>(p.codes)[u] = c;
        // a word of scales is four blocks, sixteen lanes; blocks past the row's end have a scale of one
        const uint32_t block = at[i] / 4, words = (p.per_row + 15) / 16;
        if (at[i] % 4 == 0) {
            uint8_t* s = p.scales + static_cast<int64_t>(row[i]) * (4 * words) + block;
            *s = static_cast<uint8_t>(e);
            if (at[i] + 4 == p.per_row)
                for (uint32_t b = block + 1; b < 4 * words; ++b) s[b - block] = 127;
        }
    }
}

template <bool kVec>
__global__ void __launch_bounds__(kThreads) act8_load_kernel(const Act8Params p) {
    pdl_wait();
    pdl_trigger();
    const uint32_t u0 = blockIdx.x * (kThreads * kUnits) + threadIdx.x;
    const uint32_t words = (p.per_row + 15) / 16;
    uint2 c[kUnits];
    uint32_t row[kUnits], at[kUnits], e[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t u = u0 + i * kThreads;
        row[i] = u / p.per_row;
        at[i] = u - row[i] * p.per_row;
        c[i] = make_uint2(0u, 0u);
        e[i] = 127;
        if (u < p.units) {
            c[i] = __ldcs(reinterpret_cast<const uint2*>(p.codes) + u);
            e[i] = p.scales[static_cast<int64_t>(row[i]) * (4 * words) + at[i] / 4];
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        if (u0 + i * kThreads >= p.units) continue;
        const float scale = act8_scale(e[i]);
        float a[4], b[4];
        act8_decode4(c[i].x, scale, a);
        act8_decode4(c[i].y, scale, b);
        store_unit<kVec>(p.x + row[i] * p.ld, static_cast<int>(at[i]) * 8, p.width,
                         make_uint4(exact_bf16x2(a[0], a[1]), exact_bf16x2(a[2], a[3]), exact_bf16x2(b[0], b[1]),
                                    exact_bf16x2(b[2], b[3])));
    }
}

dim3 grid_of(const Act8Params& p) { return dim3((p.units + kThreads * kUnits - 1) / (kThreads * kUnits)); }

}  // namespace

cudaError_t launch_act8_store(const Act8Params& p, cudaStream_t stream) {
    return launch_pdl(p.vector ? act8_store_kernel<true> : act8_store_kernel<false>, grid_of(p), dim3(kThreads), 0, stream, p);
}

cudaError_t launch_act8_load(const Act8Params& p, cudaStream_t stream) {
    return launch_pdl(p.vector ? act8_load_kernel<true> : act8_load_kernel<false>, grid_of(p), dim3(kThreads), 0, stream, p);
}

}  // namespace lora
