// Rotary positions on queries and keys, and keys and values into the rows of a cache.
//
//   pair i of a head at position t:  (a, b) -> m (a cos - b sin, b cos + a sin) of the angle t f_i;  backward: of -t f_i
//
// Pairs are (x_i, x_{i + rot/2}) or, interleaved, (x_{2i}, x_{2i+1}) of a head's first `rot` features; the rest is copied.
// Angles are turns in 64-bit fixed point: t times the turns a position, modulo 2^64, is exact up to the rounding of that
// factor (2^-65 of a turn a position), so far positions lose nothing where fp32 products would be off by radians.
//
// Bound by memory.  A unit is two vectors of 16 bytes of a head: eight pairs, or two vectors to copy.  A head's units lie in consecutive
// lanes, g heads side by side, and a warp works on an item: up to 4 g heads of Q, 2 g of K and of V of one row, then on another item.
// So a lane's places in a head are formed once and its eight sines and cosines once an item (each pair's by one lane, shared through
// shared memory), and an item's loads, up to sixteen vectors a lane, are under way together.  8192 rows of 40 heads of 128 (168 MB) take
// 33 us, 5.1 TB/s; 42 where a lane's units lay anywhere in a row, 36 with a row a warp.
#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.h"
#include "rope.h"

#include <type_traits>

namespace lora {

namespace {

constexpr int kWarps = 4;
constexpr int kQHeads = kRopeQHeads, kKHeads = kRopeKHeads;   // of a lane, at most
// CTAs of an SM: 128 registers a thread (the widest form spills 16 bytes), 168 with V.  Fewer spill more: 8192 rows of 40 heads 38 us with five CTAs, 33 with four;
// 5000 rows into a cache 20 us with four, 18 with three.
constexpr int ctas_of(bool append) { return append ? 3 : 4; }

template <int W> struct Vec;
template <> struct Vec<8> { using type = uint4; };
template <> struct Vec<4> { using type = uint2; };
template <> struct Vec<2> { using type = uint32_t; };
template <> struct Vec<1> { using type = uint16_t; };

template <int W>
union Pack {
    typename Vec<W>::type v;
    uint16_t x[W];
    uint32_t w[W < 2 ? 1 : W / 2];
};

__device__ __forceinline__ float wide(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

__device__ __forceinline__ F2 wide2(uint32_t w) { return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
__device__ __forceinline__ uint32_t narrow2(F2 v) {
    const float2 x = parts(v);
    return pack_bf16x2(x.x, x.y);
}

// The sines and cosines of a lane's W pairs; without interleaving two neighbours side by side.
template <int W, bool kInter>
struct Turn {
    F2 c[W < 2 ? 1 : W / 2], s[W < 2 ? 1 : W / 2];
    __device__ __forceinline__ void load(const float2* cs) {
        if (W == 1) {
            c[0] = f2(cs[0].x, 0.f);
            s[0] = f2(cs[0].y, 0.f);
        } else {
#pragma unroll
            for (int k = 0; k < W / 2; ++k) {
                const float4 q = reinterpret_cast<const float4*>(cs)[k];
                c[k] = f2(q.x, q.z);
                s[k] = f2(q.y, q.w);
            }
        }
    }
    // (a, b) -> (a c - b s, b c + a s)
    __device__ __forceinline__ void apply(Pack<W>& a, Pack<W>& b) const {
        if (W == 1) {
            const float f = wide(a.x[0]), g = wide(b.x[0]), x = parts(c[0]).x, y = parts(s[0]).x;
            const uint32_t r = pack_bf16x2(f * x - g * y, g * x + f * y);
            a.x[0] = static_cast<uint16_t>(r);
            b.x[0] = static_cast<uint16_t>(r >> 16);
        } else if (kInter) {
#pragma unroll
            for (int k = 0; k < W; ++k) {   // word k of the two vectors is pair k
                uint32_t& word = k < W / 2 ? a.w[k < W / 2 ? k : 0] : b.w[k < W / 2 ? 0 : k - W / 2];
                const float2 cc = parts(c[k / 2]), ss = parts(s[k / 2]);
                const float x = k & 1 ? cc.y : cc.x, y = k & 1 ? ss.y : ss.x;
                const float f = __uint_as_float(word << 16), g = __uint_as_float(word & 0xFFFF0000u);
                word = pack_bf16x2(f * x - g * y, g * x + f * y);
            }
        } else {
#pragma unroll
            for (int k = 0; k < W / 2; ++k) {
                const F2 f = wide2(a.w[k]), g = wide2(b.w[k]), minus = f2(-parts(s[k]).x, -parts(s[k]).y);
                a.w[k] = narrow2(fma2(f, c[k], mul(g, minus)));
                b.w[k] = narrow2(fma2(g, c[k], mul(f, s[k])));
            }
        }
    }
};

// A lane's units of up to N heads, every g-th from its first one on.
template <int W, int N>
struct Run {
    using V = typename Vec<W>::type;
    Pack<W> a[N], b[N];
    uint16_t* y;
    int64_t step;         // from one of its heads to the next in y
    int n, second;        // units; from a unit's first vector to its second (0: none)

    // heads [h0, h1) of `in` and `out`, which go to row `to`; `sub`: the lane's first of them; from: its place in a head
    __device__ __forceinline__ void load(const RopeMat& in, const RopeMat& out, int64_t row, int64_t to, int h0, int h1, int sub, int g,
                                         bool has, int from, int more) {
        n = has ? h1 - h0 - sub : 0;
        second = more;
        const uint16_t* x = in.p + row * in.row + (h0 + sub) * in.head + from;
        y = out.p + to * out.row + (h0 + sub) * out.head + from;
        step = g * out.head;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i * g >= n) break;
            a[i].v = *reinterpret_cast<const V*>(x + i * g * in.head);
            b[i].v = *reinterpret_cast<const V*>(x + i * g * in.head + more);
        }
    }
    template <bool kInter>
    __device__ __forceinline__ void store(int g, bool turn, const Turn<W, kInter>& by) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i * g >= n) break;
            if (turn) by.apply(a[i], b[i]);
            *reinterpret_cast<V*>(y + i * step) = a[i].v;
            if (second) *reinterpret_cast<V*>(y + i * step + second) = b[i].v;
        }
    }
};

template <int W, bool kInter, bool kAppend>
__global__ void __launch_bounds__(kWarps * 32, ctas_of(kAppend)) rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ __align__(16) float2 table[kWarps][kRopeMaxPairs];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t all = static_cast<uint32_t>(p.rows) * p.items, stride = gridDim.x * kWarps;
    float2* cs = table[warp];
    const int lane_sub = p.each >= 32 ? 0 : lane / p.each, lane_u = lane - lane_sub * p.each;
    const auto position = [&](uint32_t row) {
        return p.positions64 ? static_cast<const int64_t*>(p.positions)[row] : static_cast<const int32_t*>(p.positions)[row];
    };
    const auto slot = [&](uint32_t row) { return kAppend ? p.slots[row] : static_cast<int64_t>(row); };
    uint32_t item = blockIdx.x * kWarps + warp;
    if (item >= all) return;
    // items go on by `stride`: so many rows, and so many items of a row
    const uint32_t step_rows = stride / p.items;
    const int step_j = static_cast<int>(stride - step_rows * p.items);
    uint32_t row = item / p.items;
    int j = static_cast<int>(item - row * p.items);
    int64_t t = position(row), to = slot(row);
    // the turns of this lane's pairs (in registers: lanes that read a parameter at different places do so one after the other)
    uint64_t turn_of[kRopeMaxPairs / 32];
#pragma unroll
    for (int i = 0; i < kRopeMaxPairs / 32; ++i) turn_of[i] = 32 * i < p.rot / 2 ? p.turn[32 * i + lane] : 0;
    for (; item < all; item += stride) {
        const bool stored = !kAppend || (to >= 0 && to < p.slot_rows);
        // the item's heads of Q, and of K and V
        const int q0 = p.q_each * j, q1 = min(q0 + p.q_each, p.q_heads), k0 = p.k_each * j, k1 = min(k0 + p.k_each, p.kv_heads);
        uint32_t next_row = row + step_rows;
        int next_j = j + step_j;
        if (next_j >= p.items) {
            next_j -= p.items;
            ++next_row;
        }
        int64_t next_t = 0, next_to = 0;
        for (int u0 = 0; u0 < p.each; u0 += 32) {   // once, but for narrow vectors of large heads
            const int sub = lane_sub, u = u0 + lane_u;
            const bool active = sub < p.g && u < p.each, turn = u < p.units;
            // two vectors: pairs to turn, or two to copy (the second may be missing)
            int at = kInter ? 2 * u * W : u * W, second = kInter ? W : p.rot / 2;
            if (!turn) {
                at = p.rot + 2 * (u - p.units) * W;
                second = at + W < p.d ? W : 0;
            }
            Run<W, kQHeads> q;
            Run<W, kKHeads> k, v;
            q.load(p.q, p.qo, row, row, q0, q1, sub, p.g, active && (turn || u < p.units + p.q_copies), at, second);
            k.load(p.k, p.ko, row, to, k0, k1, sub, p.g, active && stored && (turn || u < p.units + p.k_copies), at, second);
            if (kAppend) v.load(p.v, p.vo, row, to, k0, k1, sub, p.g, active && stored && u < p.v_units, 2 * u * W, (2 * u + 1) * W < p.d ? W : 0);
            if (u0 == 0) {
                if (item + stride < all) {
                    next_t = position(next_row);
                    next_to = slot(next_row);
                }
                __syncwarp();   // the item before is done with the table
#pragma unroll
                for (int i = 0; i < kRopeMaxPairs / 32; ++i) {
                    if (32 * i >= p.rot / 2) break;
                    const uint64_t turns = static_cast<uint64_t>(t) * turn_of[i];
                    // signed, in half turns: [-1, 1)
                    const float half = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 4.656612873077393e-10f;
                    float s, c;
                    sincospif(half, &s, &c);
                    cs[32 * i + lane] = make_float2(c * p.magnitude, (p.back ? -s : s) * p.magnitude);
                }
                __syncwarp();
            }
            Turn<W, kInter> by;
            if (turn && active) by.load(cs + u * W);
            q.store(p.g, turn, by);
            k.store(p.g, turn, by);
            if (kAppend) v.store(p.g, false, by);
        }
        row = next_row;
        j = next_j;
        t = next_t;
        to = next_to;
    }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int W, int sms, cudaStream_t stream) {
    const int64_t items = static_cast<int64_t>(p.rows) * p.items;
    const dim3 grid(static_cast<uint32_t>(std::min<int64_t>((items + kWarps - 1) / kWarps, sms * ctas_of(p.slots != nullptr)))), block(kWarps * 32);
    const auto form = [&p](auto append) {
        constexpr bool A = decltype(append)::value;
        return [&p](int w) {
            return w == 8 ? (p.interleaved ? rope_kernel<8, true, A> : rope_kernel<8, false, A>)
                 : w == 4 ? (p.interleaved ? rope_kernel<4, true, A> : rope_kernel<4, false, A>)
                 : w == 2 ? (p.interleaved ? rope_kernel<2, true, A> : rope_kernel<2, false, A>)
                          : (p.interleaved ? rope_kernel<1, true, A> : rope_kernel<1, false, A>);
        };
    };
    auto* k = p.slots ? form(std::true_type())(W) : form(std::false_type())(W);
    return launch_pdl(k, grid, block, 0, stream, p);
}

}  // namespace lora
