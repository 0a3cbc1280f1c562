// One AdamW step over many tensors at once.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// Bound by memory: every state is read and written once, 16 bytes at a time (22 bytes a bf16 value with fp32 states,
// 10 with 8-bit states).  A CTA works on one chunk of consecutive values of one tensor; the table of tensors is a kernel
// parameter that the CTA searches for its chunk.
//
// 8-bit states: m and sqrt(v) in e4m3, 256 values with one fp32 scale (largest value / 448).  sqrt(v) has half the
// exponent range of v, and a positive one is never rounded to zero (the smallest code stands in): the step of a value
// whose v is far below its block's largest stays bounded by that code instead of growing to m / eps.  The update uses
// the new states before they are rounded.  The states' arithmetic is one IEEE rounding an operation, in the order
// written, with no contraction: which code a value gets does not depend on the compiler.
#include "adamw.h"
#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.h"

namespace lora {

namespace {

constexpr int kT = 256;
constexpr int kPer = 8;                                // values of a lane: 16 bytes of bf16
template <bool B8>
constexpr int kRounds = (B8 ? kAdamChunk8 : kAdamChunk32) / (kT * kPer);
static_assert(kPer * 32 == kAdamBlock, "a warp holds one block of the 8-bit states");
constexpr float kE4m3Max = 448.f;
constexpr float kSmallest = 0.001953125f;              // 2^-9, e4m3's smallest positive value
constexpr float kTiny = 7.888609052210118e-31f;        // 2^-100: a block below this is held as zeros

// Eight values of a lane as they lie in memory, bf16 or fp32 (with `left` < 8 the rest is zero).
template <bool kF32>
struct Raw8 {
    uint4 v[kF32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* p, int64_t at, int left) {
        if (left >= 8) {
#pragma unroll
            for (int i = 0; i < (kF32 ? 2 : 1); ++i)
                v[i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + at * (kF32 ? 4 : 2)) + i);
            return;
        }
        uint32_t w[kF32 ? 8 : 4];
#pragma unroll
        for (int i = 0; i < (kF32 ? 8 : 4); ++i) w[i] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) {
                if (kF32) w[i] = static_cast<const uint32_t*>(p)[at + i];
                else w[i / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p)[at + i]) << (16 * (i & 1));
            }
#pragma unroll
        for (int i = 0; i < (kF32 ? 2 : 1); ++i) v[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    __device__ __forceinline__ void get(F2 (&x)[4]) const {
        if (kF32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 q = v[kF32 ? i : 0];
                x[2 * i] = f2(__uint_as_float(q.x), __uint_as_float(q.y));
                x[2 * i + 1] = f2(__uint_as_float(q.z), __uint_as_float(q.w));
            }
        } else {
            const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
        }
    }
};

template <bool f32>
__device__ __forceinline__ void store8(void* p, int64_t at, int left, const F2 (&pairs)[4]) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 q = parts(pairs[i]);
        x[2 * i] = q.x;
        x[2 * i + 1] = q.y;
    }
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

// 1 / x to 2^-22; x is at least eps, a normal number.
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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

__device__ __forceinline__ uint2 load_codes(const void* codes, int64_t at, int left) {
    const uint8_t* p = static_cast<const uint8_t*>(codes);
    if (left >= 8) return __ldcs(reinterpret_cast<const uint2*>(p + at));
    uint2 c = make_uint2(0u, 0u);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) {
            if (i < 4) c.x |= static_cast<uint32_t>(p[at + i]) << (8 * i);
            else c.y |= static_cast<uint32_t>(p[at + i]) << (8 * (i - 4));
        }
    return c;
}
__device__ __forceinline__ void decode(uint2 c, float scale, F2 (&x)[4]) {
    const uint32_t w[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = from_e4m3(w[i]);
        x[i] = mul(f2(f.x, f.y), f2(scale, scale));
    }
}

// The largest |x| of two values and a third, a NaN if one is there.
__device__ __forceinline__ float max_abs(float t, float2 x) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(t), "f"(fabsf(x.x)), "f"(fabsf(x.y)));
    return r;
}

// One block (this warp's 256 values; x is 0 past the tensor's end) in 8 bits.  kPositive: x is not negative.  An infinite
// or NaN value gets the NaN code and has no part in the scale: the rest of its block keeps its states.
template <bool kPositive>
__device__ __forceinline__ void store_codes(uint8_t* p, float* scale, int64_t at, int left, F2 (&x)[4]) {
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) most = max_abs(most, parts(x[i]));
    // the sign is clear: values order like their bits, infinity and NaN above the rest
    float top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most)));
    if (__float_as_uint(top) >= 0x7F800000u) {   // in the whole warp alike; 1.3 us of the 94 of a model's adapters
        most = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = fma2(x[i], f2(0.f, 0.f), x[i]);   // infinities become NaN: their conversion is the largest code
            const float2 q = parts(x[i]);
            most = fmaxf(most, fmaxf(fabsf(q.x), fabsf(q.y)));   // a NaN counts for nothing
        }
        top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most)));
    }
    if (top < kTiny) top = 0.f;
    const float f = top > 0.f ? __fmul_rn(__frcp_rn(top), kE4m3Max) : 0.f;
    float2 y[4];
    float least = kE4m3Max;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[i] = parts(mul(x[i], f2(f, f)));
        if (kPositive) least = fminf(least, fminf(y[i].x, y[i].y));
    }
    // rare: a value below the smallest code (and the zeros, which stay zeros)
    if (kPositive && least < kSmallest && top > 0.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 q = parts(x[i]);
            if (q.x > 0.f) y[i].x = fmaxf(y[i].x, kSmallest);
            if (q.y > 0.f) y[i].y = fmaxf(y[i].y, kSmallest);
        }
    }
    const uint2 c = make_uint2(to_e4m3(y[0].x, y[0].y) | (to_e4m3(y[1].x, y[1].y) << 16),
                               to_e4m3(y[2].x, y[2].y) | (to_e4m3(y[3].x, y[3].y) << 16));
    if (left >= 8) {
        __stcs(reinterpret_cast<uint2*>(p + at), c);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[at + i] = static_cast<uint8_t>((i < 4 ? c.x >> (8 * i) : c.y >> (8 * (i - 4))) & 0xFFu);
    }
    if (lane_id() == 0) *scale = __fmul_rn(top, 1.f / kE4m3Max);
}

// What one round of a lane reads.
template <bool PF, bool GF, bool B8, bool MA>
struct Loads {
    Raw8<GF> g;
    Raw8<PF || MA> p;
    Raw8<true> m, v;           // fp32 states
    uint2 mc, vc;              // 8-bit states
    float ms, vs;
    __device__ __forceinline__ void load(const AdamTensor& t, int64_t at, int left) {
        g.load(t.grad, at, left);
        p.load(MA ? t.master : t.param, at, left);
        if (B8) {
            mc = load_codes(t.m, at, left);
            vc = load_codes(t.v, at, left);
            const int64_t block = at / kAdamBlock;   // of the warp's first lane: inside the tensor
            ms = t.m_scale[block];
            vs = t.v_scale[block];
        } else {
            m.load(t.m, at, left);
            v.load(t.v, at, left);
        }
    }
};

// The CTA's chunk: the loads of the next round are in flight while this one is worked on.
template <bool PF, bool GF, bool B8, bool MA>
__device__ __forceinline__ void chunk_step(const AdamStep& s, const AdamTensor& t, int64_t first, float gs) {
    Loads<PF, GF, B8, MA> in, next;
    const int64_t warp_first = first - static_cast<int64_t>(lane_id()) * kPer;
    const auto left_at = [&](int r) {
        return static_cast<int>(min(max(t.n - first - static_cast<int64_t>(r) * kT * kPer, int64_t{0}), int64_t{8}));
    };
    // whole warps leave together: a block of the 8-bit states is one warp's
    const auto there = [&](int r) {
        return r < kRounds<B8> && warp_first + static_cast<int64_t>(r) * kT * kPer < t.n;
    };
    if (!there(0)) return;
    in.load(t, first, left_at(0));
#pragma unroll
    for (int r = 0; r < kRounds<B8>; ++r) {
        const int64_t at = first + static_cast<int64_t>(r) * kT * kPer;
        const int left = left_at(r);
        const bool more = there(r + 1);
        if (more) next.load(t, at + kT * kPer, left_at(r + 1));
        F2 p[4], g[4], m[4], v[4], root[4];
        in.g.get(g);
        in.p.get(p);
        if (B8) {
            decode(in.mc, in.ms, m);
            decode(in.vc, in.vs, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = mul(v[i], v[i]);
        } else {
            in.m.get(m);
            in.v.get(v);
        }
        const F2 b1 = f2(s.b1, s.b1), b1c = f2(s.b1c, s.b1c), b2 = f2(s.b2, s.b2), b2c = f2(s.b2c, s.b2c);
        // sums as x 1 + y: a packed product and a packed sum would be contracted into one rounding
        const F2 one = f2(s.one, s.one);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            g[i] = mul(g[i], f2(gs, gs));
            m[i] = fma2(mul(m[i], b1), one, mul(g[i], b1c));
            v[i] = fma2(mul(v[i], b2), one, mul(mul(g[i], g[i]), b2c));
            const float2 q = parts(v[i]);
            root[i] = f2(__fsqrt_rn(q.x), __fsqrt_rn(q.y));
            const float2 d = parts(fma2(root[i], f2(s.inv_c2, s.inv_c2), f2(s.eps, s.eps)));
            p[i] = fma2(mul(m[i], f2(s.rate, s.rate)), f2(rcp(d.x), rcp(d.y)), mul(p[i], f2(s.keep, s.keep)));
        }
        if (MA) store8<true>(t.master, at, left, p);
        store8<PF>(t.param, at, left, p);
        if (B8) {
            const int64_t block = at / kAdamBlock;
            store_codes<false>(static_cast<uint8_t*>(t.m), t.m_scale + block, at, left, m);
            store_codes<true>(static_cast<uint8_t*>(t.v), t.v_scale + block, at, left, root);
        } else {
            store8<true>(t.m, at, left, m);
            store8<true>(t.v, at, left, v);
        }
        if (!more) break;
        in = next;
    }
}

// kB8: the launch's tensors have 8-bit states, else fp32 ones.  Measured (cold caches) on every adapter of a 32-layer model at rank
// 16 (8-bit) and on 207 M values with an fp32 copy: four CTAs an SM and chunks of 4096 against three and 2048 take
// 94 against 112 us with 8-bit states (bound by issue slots), 852 against 836 us with fp32 ones (bound by HBM, 7.0 TB/s).
// Back to back, with states in L2, the 8-bit step takes 87 us.
template <bool kB8, int N>
__global__ void __launch_bounds__(kT, kB8 ? 4 : 3) adamw_kernel(const __grid_constant__ AdamStep s, const __grid_constant__ AdamTensors<N> table) {
    pdl_wait();
    pdl_trigger();
    int lo = 0, hi = s.n;   // the last tensor whose first chunk is not after this one
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (table.chunk0[mid] <= static_cast<int>(blockIdx.x)) lo = mid;
        else hi = mid;
    }
    const AdamTensor& t = table.t[lo];
    const int64_t first = static_cast<int64_t>(static_cast<int>(blockIdx.x) - table.chunk0[lo]) *
                              (kB8 ? kAdamChunk8 : kAdamChunk32) + threadIdx.x * kPer;
    const float gs = s.grad_scale ? *s.grad_scale : 1.f;
    const bool gf = t.flags & kAdamGradF32;
    if (t.flags & kAdamParamF32) gf ? chunk_step<true, true, kB8, false>(s, t, first, gs) : chunk_step<true, false, kB8, false>(s, t, first, gs);
    else if (t.master) gf ? chunk_step<false, true, kB8, true>(s, t, first, gs) : chunk_step<false, false, kB8, true>(s, t, first, gs);
    else gf ? chunk_step<false, true, kB8, false>(s, t, first, gs) : chunk_step<false, false, kB8, false>(s, t, first, gs);
}

template <bool kB8>
cudaError_t run(const AdamStep& p, const AdamTensors<kAdamTensors>& t, int chunks, cudaStream_t stream) {
    if (p.n > kAdamFew) return launch_pdl(adamw_kernel<kB8, kAdamTensors>, dim3(chunks), dim3(kT), 0, stream, p, t);
    AdamTensors<kAdamFew> few;
    for (int i = 0; i < p.n; ++i) {
        few.t[i] = t.t[i];
        few.chunk0[i] = t.chunk0[i];
    }
    return launch_pdl(adamw_kernel<kB8, kAdamFew>, dim3(chunks), dim3(kT), 0, stream, p, few);
}

}  // namespace

cudaError_t launch_adamw(const AdamStep& p, const AdamTensors<kAdamTensors>& t, bool bits8, int chunks, cudaStream_t stream) {
    return bits8 ? run<true>(p, t, chunks, stream) : run<false>(p, t, chunks, stream);
}

}  // namespace lora
