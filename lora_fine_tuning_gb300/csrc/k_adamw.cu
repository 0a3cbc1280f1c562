// One AdamW step over many tensors at once.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// Bound by memory: every state is read and written once, 16 bytes at a time (22 bytes a bf16 value with fp32 states,
// 10 with 8-bit states).  A CTA works on 4096 consecutive values of one tensor; the table of tensors is a kernel
// parameter that the CTA searches for its chunk.
//
// 8-bit states: m and sqrt(v) in e4m3, 256 values with one fp32 scale (largest value / 448).  sqrt(v) has half the
// exponent range of v, and a positive one is never rounded to zero (the smallest code stands in): the step of a value
// whose v is far below its block's largest stays bounded by that code instead of growing to m / eps.  The update uses
// the new states before they are rounded.  The states' arithmetic is one IEEE rounding an operation, in the order
// written, with no contraction: which code a value gets does not depend on the compiler.
#include "adamw.h"
#include "attn.cuh"
#include "kernels.h"

namespace lora {

namespace {

constexpr int kT = 256;
constexpr int kPer = 8;                                // values of a lane: 16 bytes of bf16
constexpr int kRounds = kAdamChunk / (kT * kPer);
static_assert(kPer * 32 == kAdamBlock, "a warp holds one block of the 8-bit states");
constexpr float kE4m3Max = 448.f;
constexpr float kTiny = 7.888609052210118e-31f;        // 2^-100: a block below this is held as zeros

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// `left` values (8 or more: all) from p at `at`, bf16 or fp32.
__device__ __forceinline__ void load8(const void* p, int64_t at, int left, bool f32, float (&x)[8]) {
    if (left >= 8) {
        if (f32) {
            const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
            const float4 a = __ldcs(q), b = __ldcs(q + 1);
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        } else {
            unpack8(__ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at)), x);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = 0.f;
        if (i < left)
            x[i] = f32 ? static_cast<const float*>(p)[at + i]
                       : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[at + i]) << 16);
    }
}

__device__ __forceinline__ void store8(void* p, int64_t at, int left, bool f32, const float (&x)[8]) {
    if (left >= 8) {
        if (f32) {
            float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
            __stcs(q, make_float4(x[0], x[1], x[2], x[3]));
            __stcs(q + 1, make_float4(x[4], x[5], x[6], x[7]));
        } else {
            __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at),
                   make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                              pack_bf16x2(x[6], x[7])));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i >= left) continue;
        if (f32) static_cast<float*>(p)[at + i] = x[i];
        else static_cast<uint16_t*>(p)[at + i] = bf16_bits(x[i]);
    }
}

// Two e4m3 codes -> two floats, and back (round to nearest even, finite values saturate).
__device__ __forceinline__ float2 from_e4m3(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
    float2 f;
    asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %2;\ncvt.f32.f16 %0, lo;\ncvt.f32.f16 %1, hi;\n}" : "=f"(f.x), "=f"(f.y) : "r"(h));
    return f;
}
__device__ __forceinline__ uint32_t to_e4m3(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void load_codes(const uint8_t* p, int64_t at, int left, float scale, float (&x)[8]) {
    uint2 c = make_uint2(0u, 0u);
    if (left >= 8) {
        c = __ldcs(reinterpret_cast<const uint2*>(p + at));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) {
                if (i < 4) c.x |= static_cast<uint32_t>(p[at + i]) << (8 * i);
                else c.y |= static_cast<uint32_t>(p[at + i]) << (8 * (i - 4));
            }
    }
    const uint32_t w[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = from_e4m3(w[i]);
        x[2 * i] = __fmul_rn(f.x, scale);
        x[2 * i + 1] = __fmul_rn(f.y, scale);
    }
}

// One block (this warp's 256 values; x is 0 past the tensor's end) in 8 bits.
template <bool kPositive>
__device__ __forceinline__ void store_codes(uint8_t* p, float* scale, int64_t at, int left, const float (&x)[8]) {
    uint32_t top_bits = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top_bits = max(top_bits, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    float top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, top_bits));   // NaN and infinity order above the rest
    if (!(top >= kTiny)) top = 0.f;
    const float f = top > 0.f ? __fmul_rn(__frcp_rn(top), kE4m3Max) : 0.f;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = __fmul_rn(x[i], f);
        if (kPositive && x[i] > 0.f && top > 0.f) y[i] = fmaxf(y[i], 0.001953125f);
    }
    const uint2 c = make_uint2(to_e4m3(y[0], y[1]) | (to_e4m3(y[2], y[3]) << 16), to_e4m3(y[4], y[5]) | (to_e4m3(y[6], y[7]) << 16));
    if (left >= 8) {
        __stcs(reinterpret_cast<uint2*>(p + at), c);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[at + i] = static_cast<uint8_t>((i < 4 ? c.x >> (8 * i) : c.y >> (8 * (i - 4))) & 0xFFu);
    }
    if (lane_id() == 0) *scale = __fmul_rn(top, 1.f / kE4m3Max);
}

template <int N>
__global__ void __launch_bounds__(kT) adamw_kernel(const __grid_constant__ AdamStep s, const __grid_constant__ AdamTensors<N> table) {
    pdl_wait();
    pdl_trigger();
    int lo = 0, hi = s.n;   // the last tensor whose first chunk is not after this one
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (table.t[mid].chunk0 <= static_cast<int>(blockIdx.x)) lo = mid;
        else hi = mid;
    }
    const AdamTensor t = table.t[lo];
    const int64_t first = static_cast<int64_t>(static_cast<int>(blockIdx.x) - t.chunk0) * kAdamChunk + threadIdx.x * kPer;
    const bool pf32 = t.flags & kAdamParamF32, gf32 = t.flags & kAdamGradF32, bits8 = t.flags & kAdam8Bit;
    const float gs = s.grad_scale ? *s.grad_scale : 1.f;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int64_t at = first + static_cast<int64_t>(r) * kT * kPer;
        // whole warps leave together: a block of the 8-bit states is one warp's
        if (at - static_cast<int64_t>(lane_id()) * kPer >= t.n) break;
        const int left = static_cast<int>(min(max(t.n - at, int64_t{0}), int64_t{8}));
        float p[8], g[8], m[8], v[8], root[8];
        load8(t.grad, at, left, gf32, g);
        if (t.master) load8(t.master, at, left, true, p);
        else load8(t.param, at, left, pf32, p);
        const int64_t block = at / kAdamBlock;
        if (bits8) {
            load_codes(static_cast<const uint8_t*>(t.m), at, left, t.m_scale[block], m);
            load_codes(static_cast<const uint8_t*>(t.v), at, left, t.v_scale[block], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], v[i]);
        } else {
            load8(t.m, at, left, true, m);
            load8(t.v, at, left, true, v);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (s.grad_scale) g[i] = __fmul_rn(g[i], gs);
            m[i] = __fadd_rn(__fmul_rn(m[i], s.b1), __fmul_rn(g[i], s.b1c));
            v[i] = __fadd_rn(__fmul_rn(v[i], s.b2), __fmul_rn(__fmul_rn(g[i], g[i]), s.b2c));
            root[i] = __fsqrt_rn(v[i]);
            const float d = fmaf(root[i], s.inv_c2, s.eps);
            p[i] = p[i] * s.keep - __fdividef(s.rate * m[i], d);
        }
        if (t.master) store8(t.master, at, left, true, p);
        store8(t.param, at, left, pf32, p);
        if (bits8) {
            store_codes<false>(static_cast<uint8_t*>(t.m), t.m_scale + block, at, left, m);
            store_codes<true>(static_cast<uint8_t*>(t.v), t.v_scale + block, at, left, root);
        } else {
            store8(t.m, at, left, true, m);
            store8(t.v, at, left, true, v);
        }
    }
}

}  // namespace

cudaError_t launch_adamw(const AdamStep& p, const AdamTensors<kAdamTensors>& t, int chunks, cudaStream_t stream) {
    if (p.n <= kAdamFew)
        return launch_pdl(adamw_kernel<kAdamFew>, dim3(chunks), dim3(kT), 0, stream, p,
                          reinterpret_cast<const AdamTensors<kAdamFew>&>(t));
    return launch_pdl(adamw_kernel<kAdamTensors>, dim3(chunks), dim3(kT), 0, stream, p, t);
}

}  // namespace lora
