// Rows that need not start on 16 bytes, read and written by aligned vectors whose lanes exchange what crosses a boundary.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace lora {

// Sixteen bytes from byte `s` (0 to 15) on of the 32 in a and b.
__device__ __forceinline__ uint4 shifted(uint4 a, uint4 b, uint32_t s) {
    uint32_t w[6] = {a.x, a.y, a.z, a.w, b.x, b.y}, x = b.z, y = b.w;
    if (s & 4) w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = w[4], w[4] = w[5], w[5] = x, x = y;
    if (s & 8) w[0] = w[2], w[1] = w[3], w[2] = w[4], w[3] = w[5], w[4] = x;
    const uint32_t r = (s & 3) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], r), __funnelshift_r(w[1], w[2], r), __funnelshift_r(w[2], w[3], r),
                      __funnelshift_r(w[3], w[4], r));
}
// The same where `s` is a multiple of two and the same in the whole warp: a branch instead of selections.
__device__ __forceinline__ uint4 shifted_alike(uint4 a, uint4 b, uint32_t s) {
    const uint32_t r = (s & 3) * 8;
    const auto words = [r](uint32_t p, uint32_t q, uint32_t u, uint32_t v, uint32_t w) {
        return make_uint4(__funnelshift_r(p, q, r), __funnelshift_r(q, u, r), __funnelshift_r(u, v, r), __funnelshift_r(v, w, r));
    };
    switch (s >> 2) {
        case 0: return words(a.x, a.y, a.z, a.w, b.x);
        case 1: return words(a.y, a.z, a.w, b.x, b.y);
        case 2: return words(a.z, a.w, b.x, b.y, b.z);
        default: return words(a.w, b.x, b.y, b.z, b.w);
    }
}
__device__ __forceinline__ uint4 shuffle_down(uint4 v) {
    return make_uint4(__shfl_down_sync(0xFFFFFFFFu, v.x, 1), __shfl_down_sync(0xFFFFFFFFu, v.y, 1),
                      __shfl_down_sync(0xFFFFFFFFu, v.z, 1), __shfl_down_sync(0xFFFFFFFFu, v.w, 1));
}
__device__ __forceinline__ uint4 shuffle_up(uint4 v) {
    return make_uint4(__shfl_up_sync(0xFFFFFFFFu, v.x, 1), __shfl_up_sync(0xFFFFFFFFu, v.y, 1),
                      __shfl_up_sync(0xFFFFFFFFu, v.z, 1), __shfl_up_sync(0xFFFFFFFFu, v.w, 1));
}

// The aligned 16 bytes at byte `at` of a row of `bytes`, zero outside the row.
template <int kSize>
__device__ __forceinline__ uint4 load_block(const uint8_t* row, int at, int bytes) {
    if (at >= 0 && at + 16 <= bytes) return __ldcs(reinterpret_cast<const uint4*>(row + at));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 16 / kSize; ++e) {
        const int b = at + e * kSize;
        if (b < 0 || b >= bytes) continue;
        if (kSize == 4) w[e & 3] = *reinterpret_cast<const uint32_t*>(row + b);
        else w[e / 2 & 3] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(row + b)) << (16 * (e & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The elements [from, to) of sixteen bytes at `x`, one by one.
template <int kSize>
__device__ __forceinline__ void store_parts(uint8_t* x, uint4 v, int from, int to) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 16 / kSize; ++e)
        if (e >= from && e < to) {
            if (kSize == 4) *reinterpret_cast<uint32_t*>(x + 4 * e) = w[kSize == 4 ? e : 0];
            else *reinterpret_cast<uint16_t*>(x + 2 * e) = static_cast<uint16_t>(w[e / 2 & 3] >> (16 * (e & 1)));
        }
}

// Sixteen bytes to byte `at` of a row of `bytes`, whose 16 bytes before have another owner's `before` (none for the first of a warp's
// share).  Where the row does not start on 16 bytes, the aligned 16 that begin in `before` are stored; the `last` of the share also
// stores the rest of its own.
// kAlike: the warp's lanes are in one row.
template <int kSize, bool kAlike>
__device__ __forceinline__ void store16(uint8_t* row, int at, int bytes, uint4 v, uint4 before, bool first, bool last) {
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u), left = bytes - at;
    if (shift == 0) {
        if (left >= 16) *reinterpret_cast<uint4*>(row + at) = v;
        else if (left > 0) store_parts<kSize>(row + at, v, 0, left / kSize);
        return;
    }
    if (!first && left + shift >= 16) {
        *reinterpret_cast<uint4*>(row + at - shift) = kAlike ? shifted_alike(before, v, 16 - shift) : shifted(before, v, 16 - shift);
    } else {
        if (!first && left + shift > 0) store_parts<kSize>(row + at - 16, before, (16 - shift) / kSize, min(16, 16 + left) / kSize);
        if (left > 0) store_parts<kSize>(row + at, v, 0, min(16 - shift, left) / kSize);
    }
    if (last && left > 16 - shift) store_parts<kSize>(row + at, v, (16 - shift) / kSize, min(16, left) / kSize);
}

}  // namespace lora
