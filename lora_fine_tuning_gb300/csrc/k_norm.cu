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
// Bound by memory.  A row is held in registers between its loads and its stores: a warp a row up to 1024 values, a CTA
// beyond.  Sums over a row are fp32, by shuffles and one exchange through shared memory; the sum of squares is formed anew
// on values 2^-80 their size where it leaves fp32's range.  The backward's sums over rows stay in a thread's registers
// over the rows that its CTA works on, and a second kernel adds the CTAs' sums in a fixed order.
#include "act8.cuh"
#include "act8.h"
#include "kernels.h"
#include "norm.h"

namespace lora {

namespace {

constexpr float kSmall = 8.271806125530277e-25f;   // 2^-80: the largest values' squares then add up far below fp32's largest

// T threads share a row, each with V units of eight values.  kVec: unit i of thread t is the columns from (i T + t) 8 on;
// else value e of unit i is column (8 i + e) T + t, so that a warp's loads are consecutive and a warp is one block in 8 bits.
template <int T, int V, bool kVec>
struct Cols {
    static __device__ __forceinline__ int at(int i, int e, int t) { return kVec ? (i * T + t) * 8 + e : (i * 8 + e) * T + t; }
};

// Eight values as they lie in memory.
template <bool kF32>
struct Unit {
    uint32_t w[kF32 ? 8 : 4];
    __device__ __forceinline__ float get(int e) const {
        if (kF32) return __uint_as_float(w[e]);
        return __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < (kF32 ? 8 : 4); ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void put(const float (&v)[8]) {
        if (kF32) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[kF32 ? e : 0] = __float_as_uint(v[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
        }
    }
};

template <int T, int V, bool kVec, bool kF32>
__device__ __forceinline__ void load_unit(Unit<kF32>& u, const void* row, int i, int t, int width) {
    u.clear();
    if (kVec) {
        const int c = (i * T + t) * 8;
        if (c >= width) return;
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + static_cast<int64_t>(c) * (kF32 ? 4 : 2));
        const uint4 a = __ldcs(q);
        u.w[0] = a.x, u.w[1] = a.y, u.w[2] = a.z, u.w[3] = a.w;
        if (kF32) {
            const uint4 b = __ldcs(q + 1);
            u.w[kF32 ? 4 : 0] = b.x, u.w[kF32 ? 5 : 0] = b.y, u.w[kF32 ? 6 : 0] = b.z, u.w[kF32 ? 7 : 0] = b.w;
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = (i * 8 + e) * T + t;
        if (c >= width) continue;
        if (kF32) u.w[kF32 ? e : 0] = static_cast<const uint32_t*>(row)[c];
        else u.w[e / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(row)[c]) << (16 * (e & 1));
    }
}

template <int T, int V, bool kVec, bool kF32>
__device__ __forceinline__ void store_unit(const Unit<kF32>& u, void* row, int i, int t, int width) {
    if (kVec) {
        const int c = (i * T + t) * 8;
        if (c >= width) return;
        uint4* q = reinterpret_cast<uint4*>(static_cast<uint8_t*>(row) + static_cast<int64_t>(c) * (kF32 ? 4 : 2));
        q[0] = make_uint4(u.w[0], u.w[1], u.w[2], u.w[3]);
        if (kF32) q[1] = make_uint4(u.w[kF32 ? 4 : 0], u.w[kF32 ? 5 : 0], u.w[kF32 ? 6 : 0], u.w[kF32 ? 7 : 0]);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = (i * 8 + e) * T + t;
        if (c >= width) continue;
        if (kF32) static_cast<uint32_t*>(row)[c] = u.w[kF32 ? e : 0];
        else static_cast<uint16_t*>(row)[c] = static_cast<uint16_t>(u.w[e / 2] >> (16 * (e & 1)));
    }
}

// Eight weights of a vector (bf16 or fp32); zero past its end.
template <int T, int V, bool kVec>
__device__ __forceinline__ void load_weights(float (&v)[8], const NormVec& w, int i, int t, int width) {
    if (w.f32) {
        if (kVec) {
            const int c = (i * T + t) * 8;
            const float4 a = c < width ? reinterpret_cast<const float4*>(static_cast<const float*>(w.p) + c)[0] : make_float4(0, 0, 0, 0);
            const float4 b = c < width ? reinterpret_cast<const float4*>(static_cast<const float*>(w.p) + c)[1] : make_float4(0, 0, 0, 0);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = (i * 8 + e) * T + t;
            v[e] = c < width ? static_cast<const float*>(w.p)[c] : 0.f;
        }
        return;
    }
    Unit<false> u;
    u.clear();
    if (kVec) {
        const int c = (i * T + t) * 8;
        if (c < width) {
            const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w.p) + c);
            u.w[0] = a.x, u.w[1] = a.y, u.w[2] = a.z, u.w[3] = a.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = (i * 8 + e) * T + t;
            if (c < width) u.w[e / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(w.p)[c]) << (16 * (e & 1));
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = u.get(e);
}

__device__ __forceinline__ float one_weight(const NormVec& w, int i) {
    return w.f32 ? static_cast<const float*>(w.p)[i]
                 : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(w.p)[i]) << 16);
}

// A row's values in 8 bits.  Whole warps take part; the row's padding up to whole blocks is zero, its scale one.
template <int T, int V, bool kVec>
__device__ __forceinline__ void store_act8(const Unit<false>& u, const NormAct8& a, const NormShape& s, int64_t row, int i, int t) {
    uint8_t* codes = a.codes + row * s.codes_ld;
    uint8_t* scales = a.scales + row * s.scales_ld;
    if (kVec) {
        const int c = (i * T + t) * 8;
        uint32_t e;
        const uint2 k = act8_encode8(make_uint4(u.w[0], u.w[1], u.w[2], u.w[3]), e);
        if (c < s.codes_ld) *reinterpret_cast<uint2*>(codes + c) = k;
        if (c % kAct8Block == 0 && c / kAct8Block < s.scales_ld) scales[c / kAct8Block] = static_cast<uint8_t>(c < s.codes_ld ? e : 127u);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = (i * 8 + j) * T + t;
        uint32_t e;
        const uint32_t k = act8_encode1((u.w[j / 2] >> (16 * (j & 1))) & 0xFFFFu, e);
        if (c < s.codes_ld) codes[c] = static_cast<uint8_t>(k);
        if (c % kAct8Block == 0 && c / kAct8Block < s.scales_ld) scales[c / kAct8Block] = static_cast<uint8_t>(c < s.codes_ld ? e : 127u);
    }
}

template <int T, int V, bool kVec>
__device__ __forceinline__ void load_act8(Unit<false>& u, const NormAct8& a, const NormShape& s, int64_t row, int i, int t) {
    const uint8_t* codes = a.codes + row * s.codes_ld;
    const uint8_t* scales = a.scales + row * s.scales_ld;
    u.clear();
    if (kVec) {
        const int c = (i * T + t) * 8;
        if (c >= s.width) return;
        const uint2 k = __ldcs(reinterpret_cast<const uint2*>(codes + c));
        const float scale = act8_scale(scales[c / kAct8Block]);
        float v[4];
        act8_decode4(k.x, scale, v);
        u.w[0] = exact_bf16x2(v[0], v[1]), u.w[1] = exact_bf16x2(v[2], v[3]);
        act8_decode4(k.y, scale, v);
        u.w[2] = exact_bf16x2(v[0], v[1]), u.w[3] = exact_bf16x2(v[2], v[3]);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = (i * 8 + j) * T + t;
        if (c >= s.width) continue;
        u.w[j / 2] |= (__float_as_uint(act8_decode1(codes[c], act8_scale(scales[c / kAct8Block]))) >> 16) << (16 * (j & 1));
    }
}

__device__ __forceinline__ void widen(Unit<false>& to, const Unit<false>& from) { to = from; }
__device__ __forceinline__ void widen(Unit<true>& to, const Unit<false>& from) {
#pragma unroll
    for (int e = 0; e < 8; ++e) to.w[e] = __float_as_uint(from.get(e));
}

// Sums over the T threads of a row, the same in each of them.  Two buffers in turn: a buffer is written again only
// after the barrier of the sum in between, which every thread passes after it has read the first.
template <int T, int N>
struct RowSums {
    float* buffer;   // 2 x N x warps, shared (unused where a warp has a row)
    int turn = 0;
    __device__ __forceinline__ explicit RowSums(float* b) : buffer(b) {}
    template <int M>
    __device__ __forceinline__ void add(float (&v)[M]) {
        static_assert(M <= N, "");
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
            for (int k = 0; k < M; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
        }
        if (T == 32) return;
        constexpr int kWarps = T / 32;
        float* b = buffer + turn * N * kWarps;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int k = 0; k < M; ++k) b[k * kWarps + (threadIdx.x >> 5)] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < M; ++k) {
            v[k] = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) v[k] += b[k * kWarps + i];
        }
    }
};

// 1 / rms from a sum of squares.
__device__ __forceinline__ float inverse_rms(float squares, const NormShape& s) { return rsqrtf(fmaf(squares, s.inv_width, s.eps)); }
__device__ __forceinline__ float inverse_rms_small(float squares, const NormShape& s) {
    return rsqrtf(fmaf(squares, s.inv_width, s.eps * kSmall * kSmall));
}
__device__ __forceinline__ bool too_large(float squares) { return !(squares < 3e38f); }

constexpr int rows_of(int T) { return T == 32 ? 4 : 1; }   // rows that a CTA works on at once

template <int T, int V, bool kVec, bool kF32>
__global__ void __launch_bounds__(T * rows_of(T)) norm_fwd_kernel(const __grid_constant__ NormFwd p) {
    constexpr int R = rows_of(T);
    __shared__ float shared[2 * (T / 32)];
    pdl_wait();
    pdl_trigger();
    const NormShape& s = p.s;
    const int t = threadIdx.x % T;
    RowSums<T, 1> sums(shared);
    for (int row = blockIdx.x * R + threadIdx.x / T; row < s.rows; row += gridDim.x * R) {
        float h[V][8];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            Unit<kF32> u;
            load_unit<T, V, kVec>(u, static_cast<const uint8_t*>(p.h) + row * p.h_ld * (kF32 ? 4 : 2), i, t, s.width);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = u.get(e);
        }
        if (p.y) {
            Unit<false> y[V];
#pragma unroll
            for (int i = 0; i < V; ++i) load_unit<T, V, kVec>(y[i], p.y + row * p.y_ld, i, t, s.width);
            float r = 1.f;
            if (s.post.p) {
                float q[1] = {0.f};
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) q[0] = fmaf(y[i].get(e), y[i].get(e), q[0]);
                sums.add(q);
                r = inverse_rms(q[0], s);
                if (too_large(q[0])) {
                    q[0] = 0.f;
#pragma unroll
                    for (int i = 0; i < V; ++i)
#pragma unroll
                        for (int e = 0; e < 8; ++e) q[0] = fmaf(y[i].get(e) * kSmall, y[i].get(e) * kSmall, q[0]);
                    sums.add(q);
                    r = inverse_rms_small(q[0], s) * kSmall;
                }
            }
            float c = s.res;
            if (s.row_gate.p) c *= one_weight(s.row_gate, row);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float f[8], w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = y[i].get(e) * r;
                if (s.post.p) {
                    load_weights<T, V, kVec>(w, s.post, i, t, s.width);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] *= w[e] + s.offset;
                }
                if (s.gate.p) {
                    load_weights<T, V, kVec>(w, s.gate, i, t, s.width);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] *= w[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i][e] = fmaf(f[e], c, h[i][e]);
                Unit<kF32> out;
                out.put(h[i]);
                store_unit<T, V, kVec>(out, static_cast<uint8_t*>(p.h_out) + row * p.h_out_ld * (kF32 ? 4 : 2), i, t, s.width);
                if (p.y8.codes) store_act8<T, V, kVec>(y[i], p.y8, s, row, i, t);
            }
        }
        if (p.h8.codes) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                Unit<false> u;
                u.put(h[i]);
                store_act8<T, V, kVec>(u, p.h8, s, row, i, t);
            }
        }
        if (!s.w.p) continue;
        float q[1] = {0.f};
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) q[0] = fmaf(h[i][e], h[i][e], q[0]);
        sums.add(q);
        float r = inverse_rms(q[0], s);
        if (too_large(q[0])) {
            q[0] = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) q[0] = fmaf(h[i][e] * kSmall, h[i][e] * kSmall, q[0]);
            sums.add(q);
            r = inverse_rms_small(q[0], s) * kSmall;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float w[8];
            load_weights<T, V, kVec>(w, s.w, i, t, s.width);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = h[i][e] * r * (w[e] + s.offset);
            Unit<false> x;
            x.put(w);
            if (p.x) store_unit<T, V, kVec>(x, p.x + row * p.x_ld, i, t, s.width);
            if (p.x8.codes) store_act8<T, V, kVec>(x, p.x8, s, row, i, t);
        }
    }
}

template <int T, int V, bool kVec, bool kF32, bool kSums>
__global__ void __launch_bounds__(T * rows_of(T)) norm_bwd_kernel(const __grid_constant__ NormBwd p) {
    constexpr int R = rows_of(T);
    __shared__ float shared[2 * 3 * (T / 32)];
    pdl_wait();
    pdl_trigger();
    const NormShape& s = p.s;
    const int t = threadIdx.x % T;
    const int group = blockIdx.x * R + threadIdx.x / T;
    const bool has_y = p.y || p.y8.codes;
    RowSums<T, 3> sums(shared);
    float sum_w[kSums ? V : 1][8], sum_k[kSums ? V : 1][8];
    if (kSums) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum_w[kSums ? i : 0][e] = sum_k[kSums ? i : 0][e] = 0.f;
    }
    for (int row = group; row < s.rows; row += gridDim.x * R) {
        Unit<kF32> dh[V];
        Unit<false> y[V];
        float d[V][8];   // the gradient of the stream
#pragma unroll
        for (int i = 0; i < V; ++i) {
            dh[i].clear();
            y[i].clear();
            if (p.dh) load_unit<T, V, kVec>(dh[i], static_cast<const uint8_t*>(p.dh) + row * p.dh_ld * (kF32 ? 4 : 2), i, t, s.width);
            if (p.y8.codes) load_act8<T, V, kVec>(y[i], p.y8, s, row, i, t);
            else if (p.y) load_unit<T, V, kVec>(y[i], p.y + row * p.y_ld, i, t, s.width);
        }
        float q[3] = {0.f, 0.f, 0.f};   // sums of h^2, t h, y^2
        if (s.post.p) {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) q[2] = fmaf(y[i].get(e), y[i].get(e), q[2]);
        }
        if (s.w.p) {
            Unit<kF32> h[V];
            Unit<false> dx[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (p.h8.codes) {
                    Unit<false> u;
                    load_act8<T, V, kVec>(u, p.h8, s, row, i, t);
                    widen(h[i], u);
                } else {
                    load_unit<T, V, kVec>(h[i], static_cast<const uint8_t*>(p.h) + row * p.h_ld * (kF32 ? 4 : 2), i, t, s.width);
                }
                load_unit<T, V, kVec>(dx[i], p.dx + row * p.dx_ld, i, t, s.width);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float w[8];
                load_weights<T, V, kVec>(w, s.w, i, t, s.width);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    d[i][e] = dx[i].get(e) * (w[e] + s.offset);
                    q[0] = fmaf(h[i].get(e), h[i].get(e), q[0]);
                    q[1] = fmaf(h[i].get(e), d[i][e], q[1]);
                }
            }
            sums.add(q);
            float r = inverse_rms(q[0], s), m = q[1] * r;
            if (too_large(q[0])) {
                float f[2] = {0.f, 0.f};
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        f[0] = fmaf(h[i].get(e) * kSmall, h[i].get(e) * kSmall, f[0]);
                        f[1] = fmaf(h[i].get(e) * kSmall, d[i][e], f[1]);
                    }
                sums.add(f);
                r = inverse_rms_small(f[0], s);
                m = f[1] * r;
                r *= kSmall;
            }
            m *= s.inv_width;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float n = h[i].get(e) * r;
                    if (kSums) sum_w[kSums ? i : 0][e] = fmaf(dx[i].get(e), n, sum_w[kSums ? i : 0][e]);
                    d[i][e] = fmaf(fmaf(-n, m, d[i][e]), r, dh[i].get(e));
                }
        } else {
            if (s.post.p) sums.add(q);
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) d[i][e] = dh[i].get(e);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            Unit<kF32> out;
            out.put(d[i]);
            store_unit<T, V, kVec>(out, static_cast<uint8_t*>(p.dh_out) + row * p.dh_out_ld * (kF32 ? 4 : 2), i, t, s.width);
        }
        if (!has_y) continue;
        float r = 1.f;
        if (s.post.p) {
            r = inverse_rms(q[2], s);
            if (too_large(q[2])) {
                float f[1] = {0.f};
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[0] = fmaf(y[i].get(e) * kSmall, y[i].get(e) * kSmall, f[0]);
                sums.add(f);
                r = inverse_rms_small(f[0], s) * kSmall;
            }
        }
        const float rg = s.row_gate.p ? one_weight(s.row_gate, row) : 1.f;
        float along[1] = {0.f};   // sum of z v
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float c[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e] = s.res;
            if (s.post.p) {
                float w[8];
                load_weights<T, V, kVec>(w, s.post, i, t, s.width);
#pragma unroll
                for (int e = 0; e < 8; ++e) c[e] *= w[e] + s.offset;
            }
            if (s.gate.p) {
                float w[8];
                load_weights<T, V, kVec>(w, s.gate, i, t, s.width);
#pragma unroll
                for (int e = 0; e < 8; ++e) c[e] *= w[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = y[i].get(e) * r;
                if (kSums) sum_k[kSums ? i : 0][e] = fmaf(d[i][e] * rg, v, sum_k[kSums ? i : 0][e]);
                d[i][e] *= c[e];
                along[0] = fmaf(d[i][e], v, along[0]);
            }
        }
        float m = 0.f;
        if (s.post.p || p.drow) {
            sums.add(along);
            if (p.drow && t == 0) p.drow[row] = along[0];
            if (s.post.p) m = along[0] * rg * s.inv_width;
        }
        if (!p.dy) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = fmaf(-(y[i].get(e) * r), m, d[i][e] * rg) * r;
            Unit<false> out;
            out.put(f);
            store_unit<T, V, kVec>(out, p.dy + row * p.dy_ld, i, t, s.width);
        }
    }
    if (kSums) {
        float* part = p.part + static_cast<int64_t>(group) * 2 * s.width;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = Cols<T, V, kVec>::at(i, e, t);
                if (c < s.width && group < p.groups) {
                    part[c] = sum_w[kSums ? i : 0][e];
                    part[s.width + c] = sum_k[kSums ? i : 0][e];
                }
            }
    }
}

// The groups' sums added in a fixed order: a warp's lanes have 32 columns, its CTA's eight warps every eighth group each.
__global__ void __launch_bounds__(256) norm_sums_kernel(const __grid_constant__ NormBwd p) {
    __shared__ float part[2][8][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, width = p.s.width;
    float a = 0.f, b = 0.f;
    if (c < width) {
        for (int g = warp; g < p.groups; g += 8) {
            a += p.part[static_cast<int64_t>(g) * 2 * width + c];
            b += p.part[(static_cast<int64_t>(g) * 2 + 1) * width + c];
        }
    }
    part[0][warp][lane] = a;
    part[1][warp][lane] = b;
    __syncthreads();
    if (warp != 0 || c >= width) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        a += part[0][i][lane];
        b += part[1][i][lane];
    }
    if (p.dw) p.dw[c] = a;
    const float w = p.s.post.p ? one_weight(p.s.post, c) + p.s.offset : 1.f;
    if (p.dgate) p.dgate[c] = p.s.res * w * b;
    if (p.dpost) p.dpost[c] = p.s.res * (p.s.gate.p ? one_weight(p.s.gate, c) : 1.f) * b;
}

// Runs f(threads, units) with the smallest of the forms that holds a row.
template <class F>
cudaError_t by_width(int width, F&& f) {
    using std::integral_constant;
    if (width <= 256) return f(integral_constant<int, 32>(), integral_constant<int, 1>());
    if (width <= 512) return f(integral_constant<int, 32>(), integral_constant<int, 2>());
    if (width <= 1024) return f(integral_constant<int, 32>(), integral_constant<int, 4>());
    if (width <= 2048) return f(integral_constant<int, 128>(), integral_constant<int, 2>());
    if (width <= 4096) return f(integral_constant<int, 256>(), integral_constant<int, 2>());
    if (width <= 8192) return f(integral_constant<int, 512>(), integral_constant<int, 2>());
    return f(integral_constant<int, 512>(), integral_constant<int, 4>());
}

}  // namespace

int norm_threads(int width) { return width <= 1024 ? 32 : width <= 2048 ? 128 : width <= 4096 ? 256 : 512; }

int norm_bwd_groups(int rows, int width, int sms) {
    const int t = norm_threads(width), r = rows_of(t), per_sm = 1024 / (t * r);
    return std::min((rows + r - 1) / r, sms * per_sm) * r;
}

cudaError_t launch_norm_fwd(const NormFwd& p, int sms, cudaStream_t stream) {
    return by_width(p.s.width, [&](auto t, auto v) {
        constexpr int T = decltype(t)::value, V = decltype(v)::value, R = rows_of(T);
        const int grid = std::min((p.s.rows + R - 1) / R, sms * (2048 / (T * R)));
        auto* k = p.s.vector ? (p.s.f32 ? norm_fwd_kernel<T, V, true, true> : norm_fwd_kernel<T, V, true, false>)
                             : (p.s.f32 ? norm_fwd_kernel<T, V, false, true> : norm_fwd_kernel<T, V, false, false>);
        return launch_pdl(k, dim3(grid), dim3(T * R), 0, stream, p);
    });
}

cudaError_t launch_norm_bwd(const NormBwd& p, int sms, cudaStream_t stream) {
    return by_width(p.s.width, [&](auto t, auto v) {
        constexpr int T = decltype(t)::value, V = decltype(v)::value, R = rows_of(T);
        const int grid = norm_bwd_groups(p.s.rows, p.s.width, sms) / R;
        auto* k = p.part ? (p.s.vector ? (p.s.f32 ? norm_bwd_kernel<T, V, true, true, true> : norm_bwd_kernel<T, V, true, false, true>)
                                       : (p.s.f32 ? norm_bwd_kernel<T, V, false, true, true> : norm_bwd_kernel<T, V, false, false, true>))
                         : (p.s.vector ? (p.s.f32 ? norm_bwd_kernel<T, V, true, true, false> : norm_bwd_kernel<T, V, true, false, false>)
                                       : (p.s.f32 ? norm_bwd_kernel<T, V, false, true, false> : norm_bwd_kernel<T, V, false, false, false>));
        return launch_pdl(k, dim3(grid), dim3(T * R), 0, stream, p);
    });
}

cudaError_t launch_norm_sums(const NormBwd& p, cudaStream_t stream) {
    return launch_pdl(norm_sums_kernel, dim3((p.s.width + 31) / 32), dim3(256), 0, stream, p);
}

}  // namespace lora
