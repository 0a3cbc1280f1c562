// Activations into 8 bits and back (act8.cuh has the format).
//
// Bound by memory: 2 + 1.03 bytes a value in either direction.  The matrix is cut into units of eight values (16 bytes of
// bf16, 8 of codes), a lane a unit and four lanes a block, so a block's largest value takes two shuffles.  A CTA has
// kUnits consecutive units a thread, its loads all under way before the first is used.  8192 x 14336 (356 MB a direction): store
// 58 us, load 48 (6.1 and 7.4 TB/s); rows that do not start on 16 bytes, read and written by exchanges between lanes, 84 and 102.
#include "act8.cuh"
#include "act8.h"
#include "kernels.h"
#include "rows.cuh"

namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;

template <bool kVec>
__global__ void __launch_bounds__(kThreads) act8_store_kernel(const Act8Params p) {
    pdl_wait();
    pdl_trigger();
    const uint32_t u0 = blockIdx.x * (kThreads * kUnits) + threadIdx.x;
    const int bytes = p.width * 2;
    const bool end_lane = (threadIdx.x & 31) == 31;
    uint4 x[kUnits], more[kVec ? 1 : kUnits];
    uint32_t row[kUnits], at[kUnits], shift[kVec ? 1 : kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t u = u0 + i * kThreads;
        row[i] = __umulhi(u, p.magic) >> p.shift;
        at[i] = u - row[i] * p.per_row;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (!kVec) more[kVec ? 0 : i] = x[i], shift[kVec ? 0 : i] = 0;
        if (u >= p.units) continue;
        const uint8_t* src = reinterpret_cast<const uint8_t*>(p.x + row[i] * p.ld);
        const int b = static_cast<int>(at[i]) * 16;
        if (kVec) {
            x[i] = load_block<2>(src, b, bytes);
        } else {
            const int s = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15u);
            shift[kVec ? 0 : i] = s;
            x[i] = load_block<2>(src, b - s, bytes);
            if (s && (end_lane || at[i] + 1 == p.per_row)) more[kVec ? 0 : i] = load_block<2>(src, b - s + 16, bytes);
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t u = u0 + i * kThreads;
        if (!kVec) {
            uint4 next = shuffle_down(x[i]);
            if (end_lane || at[i] + 1 == p.per_row) next = more[kVec ? 0 : i];
            x[i] = shifted(x[i], next, shift[kVec ? 0 : i]);
        }
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
        row[i] = __umulhi(u, p.magic) >> p.shift;
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
        const float scale = act8_scale(e[i]);
        float a[4], b[4];
        act8_decode4(c[i].x, scale, a);
        act8_decode4(c[i].y, scale, b);
        const uint4 x = make_uint4(exact_bf16x2(a[0], a[1]), exact_bf16x2(a[2], a[3]), exact_bf16x2(b[0], b[1]), exact_bf16x2(b[2], b[3]));
        const uint4 before = kVec ? x : shuffle_up(x);
        if (u0 + i * kThreads >= p.units) continue;
        const int lane = threadIdx.x & 31;
        const bool first = lane == 0 || at[i] == 0, last = lane == 31 || at[i] + 1 == p.per_row;
        uint8_t* to = reinterpret_cast<uint8_t*>(p.x + row[i] * p.ld);
        const int from = static_cast<int>(at[i]) * 16, left = p.width * 2 - from;
        if (!kVec) store16<2, false>(to, from, p.width * 2, x, before, first, last);
        else if (left >= 16) __stcs(reinterpret_cast<uint4*>(to + from), x);
        else if (left > 0) store_parts<2>(to + from, x, 0, left / 2);
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
