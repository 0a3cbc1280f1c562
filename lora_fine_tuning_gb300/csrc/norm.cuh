// Norms before and after a block, with the block's gate and its place in the stream.
//
//   rms(v) = sqrt(mean v^2 + eps),  u = y / rms(y) P (P = offset + post_w; without post_w: u = y),  C = res gate_j row_gate_t
//   h' = h + C u,   x = h' / rms(h') W   (W = offset + w)
//
// Backward, n = h' / rms(h'), v = y / rms(y) (or y):
//   t = dx W,  dh' = dh + (t - n mean(t n)) / rms(h'),   z = res gate P dh',  q = row_gate z
//   dy = (q - v mean(q v)) / rms(y)   (without post_w: q)
//   dw = sum_t dx n,  K = sum_t row_gate dh' v,  dgate = res P K,  dpost_w = res gate K,  drow_gate = sum_j z v
//
// Bound by memory.  T threads share a row (a warp up to 512 values, 512 threads up to 16384), each with V units of eight
// consecutive values.  A row comes into shared memory by asynchronous copies up to three rows ahead (one where two stages fit,
// none above 8192 values: ring_plan), a thread's own units by its own copies, so that nothing but these is waited for and a CTA's 128
// registers hold the factors W and res gate P and the backward's sums over rows instead of loads under way.  Rows are worked on in turn with one exchange over the row's threads each: what is summed
// over a row (its squares, t h, q v) is added up together with the first sums of the next row.
// Sums over a row are fp32, by pairs; the sum of squares is formed anew on values 2^-80 their size where it leaves fp32's range.
// The CTAs' sums over rows are added by a second kernel in a fixed order.
//
// Measured, 16384 x 8192 in bf16 with norms before and after and gates: forward 170 us (6.3 TB/s), backward with all
// gradients 276 us (5.8 TB/s; 499 with loads into registers and two barriers a row, 310 with the ring and two barriers).
// 8192 x 4096 without them: 48 and 67 us.
#pragma once

#include "act8.cuh"
#include "act8.h"
#include "f32x2.cuh"
#include "kernels.h"
#include "norm.h"
#include "rows.cuh"

#include <atomic>
#include <type_traits>

namespace lora {

namespace {

constexpr float kSmall = 8.271806125530277e-25f;   // 2^-80: the largest values' squares then add up far below fp32's largest

// Eight values as they lie in memory, bf16 or fp32.
template <bool kF32>
struct Unit {
    uint32_t w[kF32 ? 8 : 4];
    __device__ __forceinline__ F2 get(int i) const {   // values 2 i and 2 i + 1
        if (kF32) return f2(__uint_as_float(w[kF32 ? 2 * i : 0]), __uint_as_float(w[kF32 ? 2 * i + 1 : 0]));
        return f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    __device__ __forceinline__ void put(const F2 (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = parts(v[i]);
            if (kF32) w[kF32 ? 2 * i : 0] = __float_as_uint(x.x), w[kF32 ? 2 * i + 1 : 0] = __float_as_uint(x.y);
            else w[i] = pack_bf16x2(x.x, x.y);
        }
    }
};

__device__ __forceinline__ F2 both(float x) { return f2(x, x); }
__device__ __forceinline__ float total(F2 x) {
    const float2 p = parts(x);
    return p.x + p.y;
}

// Asynchronous copies; what lies past `valid` bytes is zero.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, int valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(valid) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t to, const void* from, int valid) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(valid) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from, int valid) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(valid) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until the last `left` groups at most are under way.
__device__ __forceinline__ void copies_wait(int left) {
    if (left <= 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (left == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 2;" ::: "memory");
}

// How a row's unit is taken from its stage: once, first of several times, or again.
enum Take { kOnce, kKeep, kPlain };

// One matrix that is read: where its rows are, and where a stage has a row's copies (both from thread t's first unit on).
// kRagged: its rows need not start on 16 bytes or be whole units.  A row is then copied by the aligned 16 bytes that it lies in, its first ones
// from before the row (inside the same 16); a warp's last lane also copies the 16 bytes after its unit, the other lanes get them
// from their neighbour.  The forms without it have none of the arithmetic for that (715 instructions a row and warp
// of the backward of 4864 x 8192, 1544 of 4864 x 8191).
// kCodes: it may be in 8 bits.
template <int T, int V, bool kF32, bool kRagged, bool kCodes>
struct Mat {
    const uint8_t* p;        // null: none
    int64_t ld;              // bytes
    const uint8_t* scales;   // in 8 bits: p has codes, which are aligned whole units
    int64_t scales_ld;
    uint32_t at;             // bytes from a stage's start
    int left;                // bytes of a row from the first unit on

    static constexpr int kSize = kF32 ? 4 : 2;
    static constexpr uint32_t kMore = V * T * 8 * kSize;   // where the last lanes' further bytes are
    __device__ __forceinline__ Mat(const void* base, int64_t ld_bytes, const NormAct8& a, const NormShape& s, uint32_t place, int t) {
        const bool codes = kCodes && a.codes != nullptr;
        scales = nullptr;
        ld = ld_bytes;
        scales_ld = s.scales_ld;
        left = (s.width - t * 8) * (codes ? 1 : kSize);
        at = place + t * (codes ? 8 : 16);
        p = static_cast<const uint8_t*>(base);
        if (codes) {
            p = a.codes + t * 8;
            scales = a.scales + t / 16 * 4;
            ld = s.codes_ld;
        } else if (!kRagged && p) {
            p += t * 8 * kSize;
        }
    }
    __device__ __forceinline__ void fetch(uint8_t* to_stage, uint32_t row, int t, int width) const {
        if (!p) return;
        const uint32_t stage = smem_u32(to_stage) + at;
        const uint8_t* x = p + static_cast<uint64_t>(ld) * row;
        if (kCodes && scales) {
            const uint8_t* y = scales + static_cast<uint64_t>(scales_ld) * row;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (left > i * T * 8) {
                    copy8(stage + i * T * 8, x + i * T * 8, 8);
                    copy4(stage + V * T * 8 - t * 4 + i * T * 4, y + i * T / 16 * 4, 4);
                }
            return;
        }
        if (!kRagged) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (left > i * T * 8 * kSize) {
                    copy16(stage + i * T * 8 * kSize, x + i * T * 8 * kSize, 16);
                    if (kF32) copy16(stage + (2 * i + 1) * T * 16, x + i * T * 32 + 16, 16);
                }
            return;
        }
        const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x)) & 15u;
        x -= shift;
        const int bytes = width * kSize + static_cast<int>(shift);
        const auto copy = [&](uint32_t to, int block) {
            const int valid = min(max(bytes - 16 * block, 0), 16);
            copy16(to, x + (valid ? 16 * block : 0), valid);
        };
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int u = i * T + t;
            if (kF32) {
                copy(stage + 2 * i * T * 16, 2 * u);
                copy(stage + (2 * i + 1) * T * 16, 2 * u + 1);
            } else {
                copy(stage + i * T * 16, u);
            }
            if (shift && (t & 31) == 31) copy(stage - t * 16 + kMore + (i * (T / 32) + t / 32) * 16, kF32 ? 2 * u + 2 : u + 1);
        }
    }
    // What no copy writes of a stage is zero from the start: the thread's units past the row's end, and all of a matrix that is not given,
    // the last lanes' further bytes among it.
    __device__ __forceinline__ void clear(uint8_t* stage) const {
        const int size = kCodes && scales ? 8 : 8 * kSize;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            uint2* x = reinterpret_cast<uint2*>(stage + at + i * T * size);
            x[0] = make_uint2(0u, 0u);
            if (!(kCodes && scales)) x[1] = make_uint2(0u, 0u);
            if (kF32 && !(kCodes && scales)) x[2 * T] = x[2 * T + 1] = make_uint2(0u, 0u);
            if (kCodes && scales) *reinterpret_cast<uint32_t*>(stage + at + V * T * 8 - threadIdx.x % T * 4 + i * T * 4) = 0u;
            if (kRagged && !p && (threadIdx.x & 31) == 31)
                *reinterpret_cast<uint4*>(stage + at - threadIdx.x % T * 16 + kMore + (i * (T / 32) + threadIdx.x % T / 32) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    // All lanes of a warp take part.
    // kKeep: a later read of the row may take the values as kPlain, aligned as this one leaves them.
    template <Take kTake>
    __device__ __forceinline__ void read(F2 (&v)[4], uint8_t* stage, uint32_t row, int i, int t) const {
        stage += at;
        if (kCodes && scales) {
            const uint2 c = *reinterpret_cast<const uint2*>(stage + i * T * 8);
            const uint32_t word = *reinterpret_cast<const uint32_t*>(stage + V * T * 8 - t * 4 + i * T * 4);
            const float scale = act8_scale((word >> (8 * ((t / 4) & 3))) & 0xFFu);
            float f[4];
            act8_decode4(c.x, scale, f);
            v[0] = f2(f[0], f[1]);
            v[1] = f2(f[2], f[3]);
            act8_decode4(c.y, scale, f);
            v[2] = f2(f[0], f[1]);
            v[3] = f2(f[2], f[3]);
            return;
        }
        Unit<kF32> u;
        uint4 a = *reinterpret_cast<const uint4*>(stage + (kF32 ? 2 * i : i) * T * 16);
        uint4 b = kF32 ? *reinterpret_cast<const uint4*>(stage + (2 * i + 1) * T * 16) : a;
        if (kRagged && kTake != kPlain) {
            const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p + static_cast<uint64_t>(ld) * row)) & 15u;
            if (shift) {
                uint4 next = shuffle_down(a);
                if ((t & 31) == 31) next = *reinterpret_cast<const uint4*>(stage - t * 16 + kMore + (i * (T / 32) + t / 32) * 16);
                if (kF32) {
                    a = shifted_alike(a, b, shift);
                    b = shifted_alike(b, next, shift);
                } else {
                    a = shifted_alike(a, next, shift);
                }
                if (kTake == kKeep) {
                    *reinterpret_cast<uint4*>(stage + (kF32 ? 2 * i : i) * T * 16) = a;
                    if (kF32) *reinterpret_cast<uint4*>(stage + (2 * i + 1) * T * 16) = b;
                }
            }
        }
        u.w[0] = a.x, u.w[1] = a.y, u.w[2] = a.z, u.w[3] = a.w;
        if (kF32) u.w[kF32 ? 4 : 0] = b.x, u.w[kF32 ? 5 : 0] = b.y, u.w[kF32 ? 6 : 0] = b.z, u.w[kF32 ? 7 : 0] = b.w;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = u.get(k);
    }
};

// All lanes of a warp take part.
template <int T, bool kF32, bool kRagged>
__device__ __forceinline__ void store_unit(const Unit<kF32>& u, void* row, int i, int t, int width) {
    uint8_t* x = static_cast<uint8_t*>(row);
    const uint4 a = make_uint4(u.w[0], u.w[1], u.w[2], u.w[3]);
    const uint4 b = kF32 ? make_uint4(u.w[kF32 ? 4 : 0], u.w[kF32 ? 5 : 0], u.w[kF32 ? 6 : 0], u.w[kF32 ? 7 : 0]) : a;
    if (!kRagged) {
        if (width - t * 8 <= i * T * 8) return;
        uint4* y = reinterpret_cast<uint4*>(x + t * (kF32 ? 32 : 16)) + i * T * (kF32 ? 2 : 1);
        y[0] = a;
        if (kF32) y[1] = b;
        return;
    }
    uint4 before = b;
    if (reinterpret_cast<uintptr_t>(x) & 15u) before = shuffle_up(b);
    const bool first = (t & 31) == 0, last = (t & 31) == 31;
    if (kF32) {
        store16<4, true>(x, (i * T + t) * 32, width * 4, a, before, first, false);
        store16<4, true>(x, (i * T + t) * 32 + 16, width * 4, b, a, false, last);
    } else {
        store16<2, true>(x, (i * T + t) * 16, width * 2, a, before, first, last);
    }
}

__device__ __forceinline__ float one_weight(const NormVec& w, int i) {
    return w.f32 ? static_cast<const float*>(w.p)[i]
                 : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(w.p)[i]) << 16);
}

// Eight weights of a vector; zero past its end.
template <int T>
__device__ __forceinline__ void load_weights(float (&v)[8], const NormVec& w, int i, int t, int width, bool vector) {
    const int c = (i * T + t) * 8;
    if (vector) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
        if (c >= width) return;
        if (w.f32) {
            const float4 a = reinterpret_cast<const float4*>(static_cast<const float*>(w.p) + c)[0];
            const float4 b = reinterpret_cast<const float4*>(static_cast<const float*>(w.p) + c)[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w.p) + c);
            const uint32_t x[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(e & 1 ? x[e / 2] & 0xFFFF0000u : x[e / 2] << 16);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < width ? one_weight(w, c + e) : 0.f;
}

// Eight factors of a row's values: offset + w, and res gate (offset + post_w).  Zero past the row's end.
template <int T>
__device__ __forceinline__ void main_factors(F2 (&f)[4], const NormShape& s, int i, int t) {
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 0.f;
    if (s.w.p) {
        load_weights<T>(w, s.w, i, t, s.width, s.vectors);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = (i * T + t) * 8 + e < s.width ? w[e] + s.offset : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = f2(w[2 * k], w[2 * k + 1]);
}
template <int T>
__device__ __forceinline__ void block_factors(F2 (&f)[4], const NormShape& s, int i, int t) {
    float v[8], w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (i * T + t) * 8 + e < s.width ? s.res : 0.f;
    if (s.post.p) {
        load_weights<T>(w, s.post, i, t, s.width, s.vectors);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= w[e] + s.offset;
    }
    if (s.gate.p) {
        load_weights<T>(w, s.gate, i, t, s.width, s.vectors);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= w[e];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = f2(v[2 * k], v[2 * k + 1]);
}

// A row's values in 8 bits.  Whole warps take part; the row's padding up to whole blocks is zero, its scale one.
template <int T>
__device__ __forceinline__ void store_act8(Unit<false> u, const NormAct8& a, const NormShape& s, uint32_t row, int i, int t) {
    uint8_t* codes = a.codes + static_cast<uint64_t>(s.codes_ld) * row;
    uint8_t* scales = a.scales + static_cast<uint64_t>(s.scales_ld) * row;
    const int c = (i * T + t) * 8;
    if (c + 8 > s.width) {   // a row of NaN leaves its padding zero, too
#pragma unroll
        for (int k = 0; k < 4; ++k) u.w[k] &= (c + 2 * k < s.width ? 0xFFFFu : 0u) | (c + 2 * k + 1 < s.width ? 0xFFFF0000u : 0u);
    }
    uint32_t e;
    const uint2 k = act8_encode8(make_uint4(u.w[0], u.w[1], u.w[2], u.w[3]), e);
    if (c < s.codes_ld) *reinterpret_cast<uint2*>(codes + c) = k;
    if (c % kAct8Block == 0 && c / kAct8Block < s.scales_ld) scales[c / kAct8Block] = static_cast<uint8_t>(c < s.codes_ld ? e : 127u);
}

// Rows that a CTA works on at once, and the CTAs of an SM: 512 threads at 128 registers.  (1024 threads of one
// unit at 64 registers spill: the backward of 16384 x 8192 takes 405 us instead of 276.)  Ten warps for rows up to 5120 values go with
// two CTAs at 96 registers: 8192 x 5120, all gradients, 136 us, where one CTA of sixteen warps takes 146, although
// the forms with sums then spill 172 to 244 bytes a thread.
constexpr int rows_of(int T) { return T >= 256 ? 1 : 256 / T; }
constexpr int per_sm(int T) { return T == 320 ? 2 : T * rows_of(T) >= 512 ? 1 : 512 / (T * rows_of(T)); }

// Sums of M values over the T threads of a row, the same in each of them.  Two buffers in turn: a buffer is written again only
// after the barrier of the sum in between, which every thread passes after it has read the first.
template <int T>
struct RowSums {
    float* buffer;   // 2 x 4 x warps of a row, shared (unused where a warp has a row)
    int barrier;     // of the row's threads
    int turn = 0;
    __device__ __forceinline__ RowSums(float* b, int id) : buffer(b), barrier(id) {}
    __device__ __forceinline__ void wait() {
        if (rows_of(T) == 1) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(barrier), "n"(T) : "memory");
    }
    // four values: after two exchanges of halves a lane has one of them, from eight lanes' shares
    __device__ __forceinline__ void add(float (&v)[4]) {
        const int lane = threadIdx.x & 31;
        const bool hi = lane & 16, mid = lane & 8;
        const float a = (hi ? v[2] : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, hi ? v[0] : v[2], 16);
        const float b = (hi ? v[3] : v[1]) + __shfl_xor_sync(0xFFFFFFFFu, hi ? v[1] : v[3], 16);
        float x = (mid ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, mid ? a : b, 8);   // lanes 8 k ..: value k
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
        if (T > 32) {
            constexpr int kWarps = T / 32;
            float* to = buffer + turn * 4 * kWarps;
            turn ^= 1;
            if ((lane & 7) == 0) to[(lane >> 3) * kWarps + threadIdx.x % T / 32] = x;
            wait();
            x = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; i += 8)
                if (i + 8 <= kWarps || (lane & 7) + i < kWarps) x += to[(lane >> 3) * kWarps + (lane & 7) + i];
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = __shfl_sync(0xFFFFFFFFu, x, 8 * k);
    }
};

// 1 / rms from a sum of squares, or from one of values 2^-80 their size (then 2^80 times as large).
__device__ __forceinline__ float inverse_rms(float squares, const NormShape& s) { return rsqrtf(fmaf(squares, s.inv_width, s.eps)); }
__device__ __forceinline__ float inverse_rms_small(float squares, const NormShape& s) {
    return rsqrtf(fmaf(squares, s.inv_width, s.eps * kSmall * kSmall));
}
__device__ __forceinline__ bool too_large(float squares) { return !(squares < 3e38f); }

// Sums of (v 2^-80)^2 and, with dx, of v 2^-80 dx W over thread t's columns t, t + T, ... of a row: for rows whose squares no fp32 holds.
template <class Row>
__device__ __noinline__ float2 small_sums(Row at, const uint16_t* dx, const NormVec w, float offset, int t, int T, int width) {
    float2 q = make_float2(0.f, 0.f);
    for (int c = t; c < width; c += T) {
        const float v = at(c) * kSmall;
        q.x = fmaf(v, v, q.x);
        if (dx) q.y = fmaf(v, __uint_as_float(static_cast<uint32_t>(dx[c]) << 16) * (one_weight(w, c) + offset), q.y);
    }
    return q;
}
template <bool kF32>
struct RowAt {
    const uint8_t *x, *scales;
    __device__ __forceinline__ float operator()(int c) const {
        if (scales) return act8_decode1(x[c], act8_scale(scales[c / kAct8Block]));
        if (kF32) return reinterpret_cast<const float*>(x)[c];
        return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(x)[c]) << 16);
    }
};

// How many of a thread's units its warp needs for a row: those of which some lane's is inside it.
template <int T, int V>
__device__ __forceinline__ int units_of(int t, int width) {
    const int first = __shfl_sync(0xFFFFFFFFu, t, 0) * 8;
    int n = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) n += i * T * 8 + first < width;
    return n;
}

// Where V units of a thread leave the registers for it, factors are kept; wider rows form them anew.
template <int T, int V>
constexpr bool kept() { return V <= 2; }

// Runs f(threads, units, ragged) with the smallest of the forms that holds a row.  Ragged rows have fewer forms: they are rare.
template <class F>
auto by_width(int width, bool ragged, F&& f) {
    using std::integral_constant;
    using Yes = std::true_type;
    using No = std::false_type;
    if (ragged) {
        if (width <= 512) return f(integral_constant<int, 32>(), integral_constant<int, 2>(), Yes());
        if (width <= 2560) return f(integral_constant<int, 160>(), integral_constant<int, 2>(), Yes());
        if (width <= 4096) return f(integral_constant<int, 256>(), integral_constant<int, 2>(), Yes());
        if (width <= 8192) return f(integral_constant<int, 512>(), integral_constant<int, 2>(), Yes());
        return f(integral_constant<int, 512>(), integral_constant<int, 4>(), Yes());
    }
    if (width <= 256) return f(integral_constant<int, 32>(), integral_constant<int, 1>(), No());
    if (width <= 512) return f(integral_constant<int, 32>(), integral_constant<int, 2>(), No());
    if (width <= 1024) return f(integral_constant<int, 64>(), integral_constant<int, 2>(), No());
    if (width <= 2048) return f(integral_constant<int, 128>(), integral_constant<int, 2>(), No());
    if (width <= 2560) return f(integral_constant<int, 160>(), integral_constant<int, 2>(), No());
    if (width <= 4096) return f(integral_constant<int, 256>(), integral_constant<int, 2>(), No());
    if (width <= 5120) return f(integral_constant<int, 320>(), integral_constant<int, 2>(), No());
    if (width <= 8192) return f(integral_constant<int, 512>(), integral_constant<int, 2>(), No());
    return f(integral_constant<int, 512>(), integral_constant<int, 4>(), No());
}

constexpr int kRingBudget = 216 * 1024;   // shared memory of an SM's rings

// CTAs of an SM and the stages of their rings (four at most), from the shared memory that a CTA's stage takes.  A second CTA is worth more
// than a third stage: 8192 x 4096 with an fp32 stream and all gradients 148 us with two CTAs of two stages, 205 with one of four.
struct RingPlan {
    int per_sm, stages;
};
RingPlan ring_plan(int cta_bytes, int most, bool kept) {
    if (!kept) return RingPlan{1, 1};   // wide rows are worked on one at a time
    for (int n = most; n > 1; --n)
        for (int stages = 4; stages >= 2; --stages)
            if (n * stages * cta_bytes <= kRingBudget) return RingPlan{n, stages};
    return RingPlan{1, std::max(2, std::min(4, kRingBudget / cta_bytes))};   // two of the largest, 8192 fp32 values, fit
}

// Bytes of a stage that a matrix takes: its units and, for ragged rows, 16 for each warp's last lane.
int stage_bytes_of(int T, int V, int size, bool ragged) { return V * T * 8 * size + (ragged ? V * (T / 32) * 16 : 0); }

// Lets a form of a kernel use the rings' shared memory, on its first launch on a device (below 64, as device_setup has it); ready: the devices that
// had one.  All 140 forms at once take 26 ms, which the first call of any operator would wait for.
template <class K>
cudaError_t let_rings(K* kernel, std::atomic<uint64_t>& ready) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    const uint64_t bit = uint64_t{1} << (device & 63);
    if (e != cudaSuccess || (ready.load(std::memory_order_acquire) & bit)) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBudget);
    if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
    return e;
}

}  // namespace

}  // namespace lora
