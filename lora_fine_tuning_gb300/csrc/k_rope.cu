// Rotary positions on queries and keys, and keys and values into the rows of a cache.
//
//   pair i of a head at position t:  (a, b) -> m (a cos - b sin, b cos + a sin) of the angle t f_i;  backward: of -t f_i
//
// Pairs are (x_i, x_{i + rot/2}) or, interleaved, (x_{2i}, x_{2i+1}) of a head's first `rot` features; the rest is copied.
// Angles are turns in 64-bit fixed point: t times the turns a position, modulo 2^64, is exact up to the rounding of that
// factor (2^-65 of a turn a position), so far positions lose nothing where fp32 products would be off by radians.
//
// Bound by memory.  A warp works on some heads of one row (all of them, or a share where there are few rows): it forms
// the row's sines and cosines once, in shared memory, and then has kBatch vectors of pairs a lane under way at a time.
#include "common.cuh"
#include "kernels.h"
#include "rope.h"

namespace lora {

namespace {

constexpr int kWarps = 4;
constexpr int kBatch = 4;

template <int W> struct Vec;
template <> struct Vec<8> { using type = uint4; };
template <> struct Vec<4> { using type = uint2; };
template <> struct Vec<2> { using type = uint32_t; };
template <> struct Vec<1> { using type = uint16_t; };

template <int W>
union Pack {
    typename Vec<W>::type v;
    uint16_t x[W];
};

__device__ __forceinline__ float wide(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

template <int W, bool kInter>
__global__ void __launch_bounds__(kWarps * 32) rope_kernel(const __grid_constant__ RopeParams p) {
    using V = typename Vec<W>::type;
    __shared__ float2 table[kWarps][kRopeMaxPairs];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const int row = static_cast<int>(item / p.chunks), chunk = static_cast<int>(item % p.chunks);
    if (row >= p.rows) return;
    float2* cs = table[warp];
    const int64_t t = p.positions64 ? static_cast<const int64_t*>(p.positions)[row] : static_cast<const int32_t*>(p.positions)[row];
    for (int i = lane; i < p.rot / 2; i += 32) {
        const uint64_t turns = static_cast<uint64_t>(t) * p.turn[i];
        // signed, in half turns: [-1, 1)
        const float half = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 4.656612873077393e-10f;
        float s, c;
        sincospif(half, &s, &c);
        cs[i] = make_float2(c * p.magnitude, (p.back ? -s : s) * p.magnitude);
    }
    __syncwarp();
    int64_t out_row = row;
    bool stored = true;
    if (p.slots) {
        out_row = p.slots[row];
        stored = out_row >= 0 && out_row < p.slot_rows;
    }
    const int heads = p.q_heads + p.kv_heads, each = p.units + p.copies;
    const int h0 = heads * chunk / p.chunks, n = (heads * (chunk + 1) / p.chunks - h0) * each;
    for (int base = lane; base < n; base += 32 * kBatch) {
        Pack<W> a[kBatch], b[kBatch];
        V *to[kBatch], *to_b[kBatch];
        int unit[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int idx = base + 32 * i;
            to[i] = to_b[i] = nullptr;
            if (idx >= n) continue;
            const int hh = each == 1 ? idx : static_cast<int>(__umulhi(static_cast<uint32_t>(idx), p.head_magic));
            const int u = idx - hh * each;
            const int h = h0 + hh;
            const bool is_q = h < p.q_heads;
            const RopeMat& in = is_q ? p.q : p.k;
            const RopeMat& out = is_q ? p.qo : p.ko;
            const int head = is_q ? h : h - p.q_heads;
            const bool turned = u < p.units;
            if (!(is_q || stored) || (!turned && !(is_q ? p.q_copies : p.k_copies))) continue;
            const int at = turned ? (kInter ? 2 * u * W : u * W) : p.rot + (u - p.units) * W;
            const int at_b = kInter ? at + W : at + p.rot / 2;
            const uint16_t* x = in.p + row * in.row + head * in.head;
            uint16_t* y = out.p + (is_q ? static_cast<int64_t>(row) : out_row) * out.row + head * out.head;
            unit[i] = u;
            a[i].v = *reinterpret_cast<const V*>(x + at);
            to[i] = reinterpret_cast<V*>(y + at);
            if (turned) {
                b[i].v = *reinterpret_cast<const V*>(x + at_b);
                to_b[i] = reinterpret_cast<V*>(y + at_b);
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (!to[i]) continue;
            if (to_b[i]) {
                uint16_t x[2 * W];
#pragma unroll
                for (int e = 0; e < W; ++e) x[e] = a[i].x[e], x[W + e] = b[i].x[e];
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    const float2 w = cs[unit[i] * W + e];
                    const int ia = kInter ? 2 * e : e, ib = kInter ? 2 * e + 1 : W + e;
                    const float u = wide(x[ia]), v = wide(x[ib]);
                    const uint32_t r = pack_bf16x2(u * w.x - v * w.y, v * w.x + u * w.y);
                    x[ia] = static_cast<uint16_t>(r);
                    x[ib] = static_cast<uint16_t>(r >> 16);
                }
#pragma unroll
                for (int e = 0; e < W; ++e) a[i].x[e] = x[e], b[i].x[e] = x[W + e];
                *to_b[i] = b[i].v;
            }
            *to[i] = a[i].v;
        }
    }
    if (!p.v_units || !stored) return;
    const int v0 = p.kv_heads * chunk / p.chunks, v1 = p.kv_heads * (chunk + 1) / p.chunks;
    for (int h = v0; h < v1; ++h)
        for (int u = lane; u < p.v_units; u += 32)
            reinterpret_cast<V*>(p.vo.p + out_row * p.vo.row + h * p.vo.head)[u] =
                reinterpret_cast<const V*>(p.v.p + row * p.v.row + h * p.v.head)[u];
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int W, int sms, cudaStream_t stream) {
    (void)sms;
    const int64_t items = static_cast<int64_t>(p.rows) * p.chunks;
    const dim3 grid(static_cast<uint32_t>((items + kWarps - 1) / kWarps)), block(kWarps * 32);
    auto* k = W == 8 ? (p.interleaved ? rope_kernel<8, true> : rope_kernel<8, false>)
              : W == 4 ? (p.interleaved ? rope_kernel<4, true> : rope_kernel<4, false>)
              : W == 2 ? (p.interleaved ? rope_kernel<2, true> : rope_kernel<2, false>)
                       : (p.interleaved ? rope_kernel<1, true> : rope_kernel<1, false>);
    return launch_pdl(k, grid, block, 0, stream, p);
}

}  // namespace lora
