// Activations in 8 bits, on the device: 32 consecutive values of a row share a power of two.
//
//   E = floor(log2 of the largest finite |x|),  scale = 2^(E - 6) (at least 2^-126),  code = round(x / scale), even on ties
//
// A power of two makes every step but the rounding exact: x / scale is exact in fp32, and code * scale is a bf16 value
// (seven bits), so that what reads codes as bf16 operands adds no rounding of its own.  Codes are whole numbers from -127 to
// 127: a bf16 value is at most 255/128 2^E, 127.5 scales, which 127 is as near to as 128.  So every value is off by
// half a scale at most, 2^-7 of its block's largest.  Code -128 holds what is not finite, as NaN.
#pragma once

#include "common.cuh"
#include "f32x2.cuh"

namespace lora {

constexpr int kAct8Block = 32;

// The scale's biased exponent from the bits of the block's largest finite bf16 |x|.
__device__ __forceinline__ uint32_t act8_exponent(uint32_t top) {
    const int e = static_cast<int>(top >> 7) - 6;
    return static_cast<uint32_t>(max(e, 1));
}

__device__ __forceinline__ float act8_scale(uint32_t exponent) { return __uint_as_float(exponent << 23); }
__device__ __forceinline__ float act8_inverse(uint32_t exponent) { return __uint_as_float((254u - exponent) << 23); }

// Two bf16 |x| at once.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The code of one bf16 value (its bits in the upper half of `x`), in the low byte; the other bytes are undefined.  The product is exact, the
// sum with 1.5 * 2^23 rounds it to a whole number, even on ties, whose bits are the sum's last.
constexpr float kAct8Magic = 12582912.f;
__device__ __forceinline__ uint32_t act8_code(uint32_t x, float inverse) {
    const float v = fminf(fmaxf(__uint_as_float(x) * inverse, -127.f), 127.f);
    return __float_as_uint(v + kAct8Magic);
}

// A finite value's largest |x| counts; the rest of a block is what holds an infinity or NaN.
__device__ __forceinline__ uint32_t finite_bits(uint32_t x16) { return (x16 & 0x7FFFu) < 0x7F80u ? x16 & 0x7FFFu : 0u; }

// Eight bf16 values of each lane -> eight codes; the four lanes that share a block (4 i .. 4 i + 3) get its scale.
// All 32 lanes take part.
__device__ __forceinline__ uint2 act8_encode8(uint4 x, uint32_t& exponent) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t t = max_u16x2(max_u16x2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), max_u16x2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    t = max_u16x2(t, __shfl_xor_sync(0xFFFFFFFFu, t, 1));
    t = max_u16x2(t, __shfl_xor_sync(0xFFFFFFFFu, t, 2));
    uint32_t top = max(t & 0xFFFFu, t >> 16);
    const bool odd = top >= 0x7F80u;   // an infinity or NaN in the block: the same in its four lanes
    if (__any_sync(0xFFFFFFFFu, odd)) {
        uint32_t f = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) f = max(f, max(finite_bits(w[i] & 0xFFFFu), finite_bits(w[i] >> 16)));
        f = max(f, __shfl_xor_sync(0xFFFFFFFFu, f, 1));
        f = max(f, __shfl_xor_sync(0xFFFFFFFFu, f, 2));
        top = f;
    }
    exponent = act8_exponent(top);
    const float inverse = act8_inverse(exponent);
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = parts(fma2(f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), f2(inverse, inverse),
                                    f2(kAct8Magic, kAct8Magic)));
        c[2 * i] = __float_as_uint(v.x);
        c[2 * i + 1] = __float_as_uint(v.y);
    }
    // only a block whose largest value has all fraction bits set holds 127.5 scales, which would round to 128
    if (__any_sync(0xFFFFFFFFu, (top & 0x7Fu) == 0x7Fu)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[2 * i] = act8_code(w[i] << 16, inverse);
            c[2 * i + 1] = act8_code(w[i] & 0xFFFF0000u, inverse);
        }
    }
    if (odd) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if ((w[i] & 0x7F80u) == 0x7F80u) c[2 * i] = 0x80u;
            if ((w[i] & 0x7F800000u) == 0x7F800000u) c[2 * i + 1] = 0x80u;
        }
    }
    uint2 out;
    out.x = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    out.y = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
    return out;
}

// Four codes -> four values, exact.  `scale` is the block's.
__device__ __forceinline__ void act8_decode4(uint32_t codes, float scale, float (&v)[4]) {
    const uint32_t u = codes ^ 0x80808080u;   // code + 128
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540u + i)) - 8388736.f) * scale;   // 2^23 + 128 + code
    const uint32_t none = (u - 0x01010101u) & ~u & 0x80808080u;   // not zero where a byte of u is zero
    if (none) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (((u >> (8 * i)) & 0xFFu) == 0u) v[i] = __int_as_float(0x7FC00000);
    }
}

__device__ __forceinline__ float act8_decode1(uint32_t code, float scale) {
    const int c = static_cast<int8_t>(code);
    return c == -128 ? __int_as_float(0x7FC00000) : static_cast<float>(c) * scale;
}

// Sixteen codes -> sixteen bf16 values, exact, without fp32 in between: a byte's low seven bits are the fraction of 128 + low (0x43..) and its
// top bit that of 128 or 256, whose difference is the code.  `scale2`: the blocks' scale in bf16, twice.
__device__ __forceinline__ uint32_t act8_scale2(uint32_t exponent) { return exponent * 0x00800080u; }
__device__ __forceinline__ uint32_t code_pair(uint32_t bytes, uint32_t scale2) {
    uint32_t r;
    asm("{\n.reg .b32 d;\nsub.rn.bf16x2 d, %1, %2;\nmul.rn.bf16x2 %0, d, %3;\n}"
        : "=r"(r) : "r"(bytes & 0xFF7FFF7Fu), "r"(bytes & 0xFF80FF80u), "r"(scale2));
    return r;
}
__device__ __forceinline__ void act8_decode16(uint4 codes, uint32_t scale2, uint4 (&v)[2]) {
    const uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w};
    uint32_t w[8], none = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[2 * i] = code_pair(__byte_perm(c[i], 0x43434343u, 0x4140), scale2);
        w[2 * i + 1] = code_pair(__byte_perm(c[i], 0x43434343u, 0x4342), scale2);
        const uint32_t u = c[i] ^ 0x80808080u;
        none |= (u - 0x01010101u) & ~u & 0x80808080u;   // not zero where a code is -128
    }
    if (none) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t two = c[i / 2] >> (16 * (i & 1));
            if ((two & 0xFFu) == 0x80u) w[i] = (w[i] & 0xFFFF0000u) | 0x7FC0u;
            if ((two & 0xFF00u) == 0x8000u) w[i] = (w[i] & 0xFFFFu) | 0x7FC00000u;
        }
    }
    v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    v[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// Four bits -> a mask of four bytes.
__device__ __forceinline__ uint32_t byte_mask(uint32_t bits) { return ((bits & 15u) * 0x00204081u & 0x01010101u) * 0xFFu; }

// Two fp32 values whose lower halves are zero -> two bf16, exact.
__device__ __forceinline__ uint32_t exact_bf16x2(float lo, float hi) {
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}

}  // namespace lora
