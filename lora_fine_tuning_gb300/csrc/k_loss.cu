// Losses on logits, forward and gradient.
//
//   logp_t = z_ty - max - log sum_v exp(z_tv - max),   d loss / d z_tv = c_t (1[v = y_t] - p_tv),   c_t = d loss / d logp_t
//
// Both losses are bound by the logits: read once, and the gradient written once.  The policy loss depends on one row
// at a time, so a row stays on chip from its one read to the write of its gradient: a short one in the registers of
// its CTA, a long one spread over the shared memory of a cluster of CTAs.  The preference loss needs the sums over
// both responses of a pair before any gradient: a pass over the logits for the statistics, the pairs' losses, and a
// pass that reads the logits again and writes the gradient.
//
// All statistics are fp32 relative to the row's maximum (p of the label is then exact to 2^-23 also near 1, where
// 1 - p is the gradient); sums over tokens are fp64 in a fixed order.

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.h"
#include "loss.h"

namespace lora {

namespace {

constexpr int kT = 512;

template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
    static constexpr int n = 8;
    static constexpr uint32_t kFill = 0xFF80FF80u;   // -inf twice
    static __device__ __forceinline__ void get(uint4 v, F2 (&x)[4]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint4 put(const F2 (&x)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 q = parts(x[i]);
            w[i] = pack_bf16x2(q.x, q.y);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // The largest of NV vectors and t (a NaN counts for nothing).
    template <int NV>
    static __device__ __forceinline__ float top(const uint4 (&v)[NV], float t) {
        uint32_t m = v[0].x;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            m = max2(m, v[k].x);
            m = max2(m, v[k].y);
            m = max2(m, v[k].z);
            m = max2(m, v[k].w);
        }
        return max3(t, __uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ float one(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
    static __device__ __forceinline__ uint16_t bits(float x) { return bf16_bits(x); }
};
template <>
struct Vec<float> {
    static constexpr int n = 4;
    static constexpr uint32_t kFill = 0xFF800000u;
    static __device__ __forceinline__ void get(uint4 v, F2 (&x)[2]) {
        x[0] = f2(__uint_as_float(v.x), __uint_as_float(v.y));
        x[1] = f2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    static __device__ __forceinline__ uint4 put(const F2 (&x)[2]) {
        const float2 a = parts(x[0]), b = parts(x[1]);
        return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
    }
    template <int NV>
    static __device__ __forceinline__ float top(const uint4 (&v)[NV], float t) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            t = max3(t, __uint_as_float(v[k].x), __uint_as_float(v[k].y));
            t = max3(t, __uint_as_float(v[k].z), __uint_as_float(v[k].w));
        }
        return t;
    }
    static __device__ __forceinline__ float one(const float* p) { return *p; }
    static __device__ __forceinline__ float bits(float x) { return x; }
};

// A row as 16-byte vectors of its memory: vector i holds elements [i n - skew, i n - skew + n).  The first and the
// last may be partial (rows of odd lengths start anywhere): those are moved element by element.
template <typename T>
struct RowView {
    const T* z;
    T* dz;
    int vocab, skew, vecs;
    bool same;   // dz's rows lie like z's: whole vectors can be stored
    __device__ __forceinline__ RowView(const LossLogits& in, int64_t row) {
        z = static_cast<const T*>(in.z) + row * in.ld;
        dz = static_cast<T*>(in.dz) + (in.dz ? row * in.dz_ld : 0);
        vocab = in.vocab;
        skew = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15u) / sizeof(T));
        vecs = (vocab + skew + Vec<T>::n - 1) / Vec<T>::n;
        same = (reinterpret_cast<uintptr_t>(dz) & 15u) / sizeof(T) == static_cast<uintptr_t>(skew);
    }
    __device__ __forceinline__ bool whole(int i) const {
        const int e = i * Vec<T>::n - skew;
        return e >= 0 && e + Vec<T>::n <= vocab;
    }
    __device__ __forceinline__ uint4 load(int i) const {
        const int e = i * Vec<T>::n - skew;
        if (i < vecs && whole(i)) return __ldcs(reinterpret_cast<const uint4*>(z + e));
        F2 x[Vec<T>::n / 2];
        const auto at = [&](int j) { return e + j >= 0 && e + j < vocab ? Vec<T>::one(z + e + j) : neg_inf(); };
#pragma unroll
        for (int j = 0; j < Vec<T>::n; j += 2) x[j / 2] = f2(at(j), at(j + 1));
        return Vec<T>::put(x);
    }
    __device__ __forceinline__ void store(int i, const F2 (&x)[Vec<T>::n / 2]) const {
        const int e = i * Vec<T>::n - skew;
        if (same && whole(i)) {
            __stcs(reinterpret_cast<uint4*>(dz + e), Vec<T>::put(x));
            return;
        }
#pragma unroll
        for (int j = 0; j < Vec<T>::n; j += 2) {
            const float2 q = parts(x[j / 2]);
            if (e + j >= 0 && e + j < vocab) dz[e + j] = Vec<T>::bits(q.x);
            if (e + j + 1 >= 0 && e + j + 1 < vocab) dz[e + j + 1] = Vec<T>::bits(q.y);
        }
    }
};

// exp(x - top); 0 for x = -inf whatever top is.
__device__ __forceinline__ float exp_from(float x, float top) { return ex2((x - top) * kLog2e); }

// exp(x - top) of a pair.
__device__ __forceinline__ F2 exp_from(F2 x, F2 minus_top) {
    const float2 q = parts(mul(add2(x, minus_top), f2(kLog2e, kLog2e)));
    return f2(ex2(q.x), ex2(q.y));
}

// The joint (maximum, sum) of all lanes' pairs, in every lane: one exponential a lane.
__device__ __forceinline__ void join_warp(float& m, float& s) {
    // floats in the order of unsigned integers
    const uint32_t bits = __float_as_uint(m);
    const uint32_t key = __reduce_max_sync(0xFFFFFFFFu, bits ^ (static_cast<uint32_t>(static_cast<int32_t>(bits) >> 31) | 0x80000000u));
    const float t = __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
    s *= exp_from(m, t);
    m = t;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
}

// c (1[v = y] - p) of one vector.
template <typename T>
__device__ __forceinline__ void grad_vec(const RowView<T>& rv, int i, uint4 raw, float top, float inv, float c, int y) {
    constexpr int n = Vec<T>::n;
    F2 x[n / 2];
    Vec<T>::get(raw, x);
    const int at = y - (i * n - rv.skew);
    const float f = -c * inv;
#pragma unroll
    for (int j = 0; j < n / 2; ++j) x[j] = mul(exp_from(x[j], f2(-top, -top)), f2(f, f));
    if (static_cast<unsigned>(at) < static_cast<unsigned>(n)) {
#pragma unroll
        for (int j = 0; j < n; j += 2)   // selects, no index: the pairs stay in registers
            x[j / 2] = add2(x[j / 2], f2(j == at ? c : 0.f, j + 1 == at ? c : 0.f));
    }
    rv.store(i, x);
}

template <typename T>
__device__ __forceinline__ void zero_vec(const RowView<T>& rv, int i) {
    F2 x[Vec<T>::n / 2];
#pragma unroll
    for (int j = 0; j < Vec<T>::n / 2; ++j) x[j] = f2(0.f, 0.f);
    rv.store(i, x);
}

// What the policy loss makes of a row's logp: its loss, and c = d loss / d logp (both without `scale`).
struct RowInputs {
    float adv, old_logp, ref;
};
__device__ __forceinline__ RowInputs row_inputs(const PolicyParams& p, int64_t row) {
    return RowInputs{p.adv[row], p.old_logp[row], p.ref ? p.ref[row] : 0.f};
}
__device__ __forceinline__ RowInputs row_inputs(const PrefParams&, int64_t) { return RowInputs{0.f, 0.f, 0.f}; }
__device__ __forceinline__ void policy_row(const PolicyParams& p, const RowInputs& in, float logp, float* loss, float* c) {
    const float a = in.adv;
    const float r = expf(logp - in.old_logp);
    const float ra = r * a;
    const float clipped = fminf(fmaxf(r, p.lo), p.hi) * a;
    const bool free = a >= 0.f ? r <= p.hi : r >= p.lo;
    float l = -fminf(ra, clipped), g = free ? -ra : 0.f;
    if (ra != ra) l = g = ra;   // fminf would drop a NaN
    if (p.ref) {
        const float x = in.ref - logp, e = expm1f(x);
        l += p.kl * (e - x);
        g -= p.kl * e;
    }
    *loss = l;
    *c = g;
}

// What a row's statistics give, by one thread: logp; the policy's loss and coefficient, or what the gradient pass of
// the preference loss reads.  Returns (maximum, 1 / sum, coefficient).
template <bool kPolicy, typename P>
__device__ __forceinline__ float3 finish_row(const P& p, int64_t row, const RowInputs& in, float top, float sum, float zy,
                                             bool write) {
    const float logp = (zy - top) - logf(sum);
    const float inv = 1.f / sum;
    float c = 0.f;
    if (write) p.in.logp[row] = logp;
    if constexpr (kPolicy) {
        float loss;
        policy_row(p, in, logp, &loss, &c);
        c *= p.scale;
        if (write) p.row_loss[row] = loss;
    } else if (write) {
        p.row[row] = LossRow{top, inv};
        p.coef[row] = 0.f;   // rows of no pair; the pairs' rows get theirs from the pairs kernel
    }
    return make_float3(top, inv, c);
}

// A row that does not count: its logits are not read.
template <bool kPolicy, typename P>
__device__ __forceinline__ void skip_row(const P& p, int64_t row) {
    p.in.logp[row] = 0.f;
    if constexpr (kPolicy) p.row_loss[row] = 0.f;
    else p.coef[row] = 0.f;
}

// The threads' (maximum, sum) of this vector group; elements past the row are -inf.
template <typename T, int NV>
__device__ __forceinline__ void group_stats(const uint4 (&v)[NV], float& m, float& s) {
    const float t = Vec<T>::top(v, m);
    s *= exp_from(m, t);
    m = t;
    F2 part[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        F2 x[Vec<T>::n / 2];
        Vec<T>::get(v[k], x);
#pragma unroll
        for (int j = 0; j < Vec<T>::n / 2; ++j) part[j & 1] = add2(part[j & 1], exp_from(x[j], f2(-t, -t)));
    }
    const float2 q = parts(add2(part[0], part[1]));
    s += q.x + q.y;
}
constexpr float kLowest = -3.402823466e+38f;   // where running maxima start: -inf - kLowest is -inf, not a NaN

template <typename T>
__device__ __forceinline__ uint4 no_vec() {
    return make_uint4(Vec<T>::kFill, Vec<T>::kFill, Vec<T>::kFill, Vec<T>::kFill);
}

// Short rows: a CTA a row, NV vectors a thread in registers.
template <typename T, int NV, bool kPolicy, typename P>
__global__ void __launch_bounds__(kT, 2) loss_rows_kernel(const __grid_constant__ P p) {
    __shared__ float2 part[kT / 32];
    __shared__ float3 result;
    pdl_wait();
    pdl_trigger();
    const int64_t row = blockIdx.x;
    const LossLogits& in = p.in;
    const RowView<T> rv(in, row);
    const int64_t y = in.labels[row];
    if (y < 0 || y >= in.vocab) {
        if (threadIdx.x == 0) skip_row<kPolicy>(p, row);
        if (kPolicy && in.dz)
            for (int i = threadIdx.x; i < rv.vecs; i += kT) zero_vec(rv, i);
        return;
    }
    uint4 v[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = k * kT + threadIdx.x;
        v[k] = i < rv.vecs ? rv.load(i) : no_vec<T>();
    }
    float zy = 0.f;
    RowInputs ri{};
    if (threadIdx.x == 0) {
        zy = Vec<T>::one(rv.z + y);
        ri = row_inputs(p, row);
    }
    float m = kLowest, s = 0.f;
    group_stats<T>(v, m, s);
    join_warp(m, s);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(m, s);
    __syncthreads();
    if (threadIdx.x < 32) {
        const float2 q = threadIdx.x < kT / 32 ? part[threadIdx.x] : make_float2(kLowest, 0.f);
        m = q.x;
        s = q.y;
        join_warp(m, s);
        if (threadIdx.x == 0) result = finish_row<kPolicy>(p, row, ri, m, s, zy, true);
    }
    if constexpr (kPolicy) {
        if (!in.dz) return;
        __syncthreads();
        const float3 r = result;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = k * kT + threadIdx.x;
            if (i < rv.vecs) grad_vec(rv, i, v[k], r.x, r.y, r.z, static_cast<int>(y));
        }
    }
}

// out = scale * sum x, in fp64 in a fixed order, by a CTA of T threads.
template <int T>
__device__ __forceinline__ void block_sum(const float* x, int64_t n, float scale, float* out) {
    __shared__ double sums[T / 32];
    double s = 0.0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < n; i += T) s += static_cast<double>(__ldcg(x + i));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < T / 32; ++w) s += sums[w];
        *out = static_cast<float>(s * static_cast<double>(scale));
    }
}

// The rows of a pair: its chosen ones, then its rejected ones.
struct PairRows {
    PrefPair q;
    __device__ __forceinline__ int count() const { return q.chosen_rows + q.rejected_rows; }
    __device__ __forceinline__ int64_t row(int i) const { return i < q.chosen_rows ? q.chosen + i : q.rejected + (i - q.chosen_rows); }
};
// What rows [from, from + step, ...) of a pair add to its margin.
__device__ __forceinline__ double margin_part(const PrefParams& p, const PairRows& pr, int from, int step) {
    double sum = 0.0;
#pragma unroll 4
    for (int i = from; i < pr.count(); i += step) {
        const int64_t r = pr.row(i), y = p.in.labels[r];
        const double d = static_cast<double>(__ldcg(p.in.logp + r)) - (p.ref ? static_cast<double>(p.ref[r]) : 0.0);
        if (y >= 0 && y < p.in.vocab) sum += i < pr.q.chosen_rows ? d : -d;
    }
    return sum;
}
// The pair's loss (without `scale`) and d (scale loss) / d margin.
__device__ __forceinline__ float2 pair_loss(const PrefParams& p, double margin) {
    const float h = static_cast<float>(static_cast<double>(p.beta) * margin);
    const float e = p.smoothing;
    // log sigmoid(h) = min(h, 0) - log1p(exp(-|h|)),  log sigmoid(-h) = log sigmoid(h) - h
    const float small = expf(-fabsf(h)), tail = log1pf(small);
    // an infinite h (a label of probability 0) leaves out the term whose weight is zero: 0 infinity would be a NaN
    const float loss = h != h ? h : (e < 1.f ? (1.f - e) * (tail - fminf(h, 0.f)) : 0.f) + (e > 0.f ? e * (tail + fmaxf(h, 0.f)) : 0.f);
    const float s_neg = (h >= 0.f ? small : 1.f) / (1.f + small);   // sigmoid(-h)
    const float s_pos = (h >= 0.f ? 1.f : small) / (1.f + small);
    const float g = h != h ? h : p.scale * p.beta * (e * s_pos - (1.f - e) * s_neg);
    return make_float2(loss, g);
}
__device__ __forceinline__ void write_coefs(const PrefParams& p, const PairRows& pr, float g, int from, int step) {
    for (int i = from; i < pr.count(); i += step) {
        const int64_t r = pr.row(i), y = p.in.labels[r];
        if (y >= 0 && y < p.in.vocab) p.coef[r] = i < pr.q.chosen_rows ? g : -g;
    }
}

// All pairs by the warps of one CTA, a warp a pair (there are no more pairs than warps), and the loss.
__device__ __forceinline__ void pairs_by_warps(const PrefLong& p, int warps) {
    const int lane = threadIdx.x & 31;
    for (int q = threadIdx.x >> 5; q < p.n_pairs; q += warps) {
        const PairRows pr{p.pairs.p[q]};
        double sum = margin_part(p, pr, lane, 32);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float2 lg = pair_loss(p, sum);
        write_coefs(p, pr, lg.y, lane, 32);
        if (lane == 0) {
            p.margin[q] = static_cast<float>(sum);
            p.pair_loss[q] = lg.x;
        }
    }
    __syncthreads();
    if (threadIdx.x >= 32) return;
    double total = 0.0;
    for (int i = lane; i < p.n_pairs; i += 32) total += static_cast<double>(__ldcg(p.pair_loss + i));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    if (lane == 0) *p.loss = static_cast<float>(total * static_cast<double>(p.scale));
}

// Long rows: a cluster of C CTAs takes rows in turn, each CTA its slice of a row.  Warps 0-15 work on a slice in
// shared memory, warp 16 keeps the ring of slices filled with bulk copies rows ahead, warp 17 sends the slice's
// statistics to the cluster's CTAs, warp 18 joins what they sent and turns it into the row's coefficient.  The
// gradient of a row is written after the statistics of the next one: the exchange runs meanwhile.  kXch exchanges can
// be under way: a CTA that sends its statistics of counted row r + 2 has finished row r, so this one has sent row r
// and finished row r - 2; its rows r - 1 to r + 2 may wait here.
//
// Both row kernels were measured (8192 rows of 128000 bf16 logits, policy loss with gradient): rows in registers of
// clusters of four take 1030 us, since a CTA neither loads while it works nor works while it loads.
constexpr int kLongThreads = kT + 96;
constexpr int kXch = 4;
constexpr int kWarps = kT / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxSlices = 8;
constexpr size_t kRingBytes = 216 * 1024;

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// 16 bytes into CTA `rank` of the cluster, counted on its barrier.
__device__ __forceinline__ void send(const float4* slot, uint64_t* bar, int rank, float4 v) {
    uint32_t a, b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(slot)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(smem_u32(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(a), "f"(v.x),
                 "f"(v.y), "f"(v.z), "f"(v.w), "r"(b)
                 : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T, bool kPolicy, typename P>
__global__ void __launch_bounds__(kLongThreads, 1)
loss_long_rows_kernel(const __grid_constant__ P p, int32_t cluster, int32_t slices, int32_t slice_bytes) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kMaxSlices], empty[kMaxSlices], part_full[2], xch[kXch], res_full[2];
    __shared__ float2 part[2][kWarps];
    __shared__ __align__(16) float4 peers[kXch][kMaxCluster];
    __shared__ float3 result[2];
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < slices; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&part_full[i], kWarps);
            mbar_init(&res_full[i], 1);
        }
        for (int i = 0; i < kXch; ++i) mbar_init(&xch[i], 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    cluster_sync();   // every CTA's barriers are there before a peer's message
    pdl_wait();
    pdl_trigger();
    const WaitCtx w{&abort_flag, p.ctl.status, p.ctl.wait_ns, kKLoss << 8};
    const LossLogits& in = p.in;
    const int64_t first = blockIdx.x / cluster, step = gridDim.x / cluster;
    const int rank = static_cast<int>(blockIdx.x % cluster);
    const bool grad = kPolicy && in.dz != nullptr;
    const auto label = [&](int64_t row) { return row < in.rows ? in.labels[row] : int64_t{-1}; };
    const auto counts = [&](int64_t y) { return y >= 0 && y < in.vocab; };

    if (warp == kWarps) {
        int n = 0;   // rows that count so far
        bool ok = true;
        int64_t y = label(first);
        for (int64_t row = first; row < in.rows; row += step) {
            const int64_t y_now = y;
            y = label(row + step);
            if (!counts(y_now)) continue;
            const RowView<T> rv(in, row);
            const int per = (rv.vecs + cluster - 1) / cluster;
            const int begin = rank * per, end = min(begin + per, rv.vecs);
            const int s = n % slices;
            ok = mbar_wait(&empty[s], ((n / slices) & 1) ^ 1u, w, 1);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            uint8_t* at = ring + static_cast<size_t>(s) * slice_bytes;
            // the row's first and last vector may reach beyond it: element by element
            int a = begin, b = end;
            T* edge = reinterpret_cast<T*>(at);
            if (a < b && !rv.whole(a)) {
                const int e = a * Vec<T>::n - rv.skew + lane;
                if (lane < Vec<T>::n) edge[lane] = e >= 0 && e < rv.vocab ? rv.z[e] : Vec<T>::bits(neg_inf());
                ++a;
            }
            if (a < b && !rv.whole(b - 1)) {
                --b;
                const int e = b * Vec<T>::n - rv.skew + lane;
                if (lane < Vec<T>::n) edge[(b - begin) * Vec<T>::n + lane] = e >= 0 && e < rv.vocab ? rv.z[e] : Vec<T>::bits(neg_inf());
            }
            __syncwarp();
            const uint32_t bytes = a < b ? static_cast<uint32_t>(b - a) * 16u : 0u;
            if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
            __syncwarp();
            // pieces of 8 KB, a lane each
            for (uint32_t o = lane * 8192u; o < bytes; o += 32u * 8192u)
                bulk_load(at + static_cast<size_t>(a - begin) * 16 + o,
                          reinterpret_cast<const uint8_t*>(rv.z + a * Vec<T>::n - rv.skew) + o, min(bytes - o, 8192u), &full[s]);
            ++n;
        }
        // every copy lands before the CTA exits, also when the warps that wait for it gave up
        if (lane == 0)
            for (int i = max(0, n - slices); i < n; ++i) mbar_wait_drain(&full[i % slices], (i / slices) & 1, p.ctl.wait_ns);
    } else if (warp == kWarps + 1) {
        int n = 0;
        int64_t y = label(first);
        float zy = lane == 0 && counts(y) ? Vec<T>::one(RowView<T>(in, first).z + y) : 0.f;
        int64_t y2 = label(first + step);
        for (int64_t row = first; row < in.rows; row += step) {
            const int64_t y_now = y;
            const float zy_now = zy;
            y = y2;
            zy = lane == 0 && counts(y) ? Vec<T>::one(RowView<T>(in, row + step).z + y) : 0.f;
            y2 = label(row + 2 * step);
            if (!counts(y_now)) continue;
            const int b = n & 1, x = n % kXch;
            bool ok = mbar_wait(&part_full[b], (n >> 1) & 1, w, 2);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const float2 q = lane < kWarps ? part[b][lane] : make_float2(kLowest, 0.f);
            float m = q.x, s = q.y;
            join_warp(m, s);
            // the label's logit goes along: with in-place gradients no peer writes the row before it was read here
            const float zs = __shfl_sync(0xFFFFFFFFu, zy_now, 0);
            if (lane < cluster) send(&peers[x][rank], &xch[x], lane, make_float4(m, s, zs, 0.f));
            ++n;
        }
    } else if (warp == kWarps + 2) {
        int n = 0;
        int64_t y = label(first);
        RowInputs ri = row_inputs(p, first);
        for (int64_t row = first; row < in.rows; row += step) {
            const int64_t y_now = y;
            const RowInputs now = ri;
            y = label(row + step);
            ri = row_inputs(p, min(row + step, in.rows - 1));
            if (!counts(y_now)) {
                if (rank == 0 && lane == 0) skip_row<kPolicy>(p, row);
                continue;
            }
            const int b = n & 1, x = n % kXch;
            if (lane == 0) mbar_arrive_expect_tx(&xch[x], static_cast<uint32_t>(cluster) * 16u);
            bool ok = mbar_wait(&xch[x], (n / kXch) & 1, w, 3);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const float4 r = lane < cluster ? peers[x][lane] : make_float4(kLowest, 0.f, 0.f, 0.f);
            float m = r.x, s = r.y;
            join_warp(m, s);
            if (lane == 0) {
                result[b] = finish_row<kPolicy>(p, row, now, m, s, r.z, rank == 0);
                mbar_arrive(&res_full[b]);
            }
            __syncwarp();
            ++n;
        }
    } else {
        int n = 0;             // rows that count so far
        int64_t prev = -1;     // the row whose gradient is due, its label and number
        int prev_y = 0;
        int64_t y = label(first);
        // one turn more than rows: the last gradient
        for (int64_t row = first;; row += step) {
            const bool more = row < in.rows;
            const int64_t y_now = y;
            if (more) y = label(row + step);
            bool due = !more;
            if (more && !counts(y_now)) {
                if (grad) {
                    const RowView<T> rv(in, row);
                    const int per = (rv.vecs + cluster - 1) / cluster;
                    const int begin = rank * per, end = min(begin + per, rv.vecs);
                    for (int i = begin + threadIdx.x; i < end; i += kT) zero_vec(rv, i);
                }
                continue;
            }
            if (more) {
                const int vecs = RowView<T>(in, row).vecs;
                const int per = (vecs + cluster - 1) / cluster;
                const int mine = min(rank * per + per, vecs) - rank * per;
                const int s = n % slices, b = n & 1;
                bool ok = mbar_wait(&full[s], (n / slices) & 1, w, 4);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const uint32_t at = smem_u32(ring) + static_cast<uint32_t>(s) * slice_bytes;
                float m = kLowest, sum = 0.f;
                for (int x = threadIdx.x; x < mine; x += 4 * kT) {
                    uint4 v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = x + k * kT < mine ? lds128(at + (x + k * kT) * 16) : no_vec<T>();
                    group_stats<T>(v, m, sum);
                }
                join_warp(m, sum);
                if (!grad) {
                    if (lane == 0) mbar_arrive(&empty[s]);
                    if (n >= 2) {   // the sending warp has read part[b] of two rows ago
                        ok = mbar_wait(&res_full[b], ((n - 2) >> 1) & 1, w, 6);
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        if (!ok) break;
                    }
                }
                if (lane == 0) {
                    part[b][warp] = make_float2(m, sum);
                    mbar_arrive(&part_full[b]);
                }
                due = n > 0;
                if (slices == 1) {   // the longest rows: the ring has no room for a row ahead
                    prev = row;
                    prev_y = static_cast<int>(y_now);
                    due = true;
                }
                ++n;
            }
            if (grad && due && prev >= 0) {
                // of counted row i: the one before this turn's, this turn's own (one slice), or the last
                const int i = more && slices > 1 ? n - 2 : n - 1;
                bool ok = mbar_wait(&res_full[i & 1], (i >> 1) & 1, w, 5);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const float3 r = result[i & 1];
                const RowView<T> rv(in, prev);
                const int per = (rv.vecs + cluster - 1) / cluster;
                const int begin = rank * per, mine = min(begin + per, rv.vecs) - begin;
                const uint32_t at = smem_u32(ring) + static_cast<uint32_t>(i % slices) * slice_bytes;
                for (int x = threadIdx.x; x < mine; x += 4 * kT) {
                    uint4 v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = x + k * kT < mine ? lds128(at + (x + k * kT) * 16) : no_vec<T>();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (x + k * kT < mine) grad_vec(rv, begin + x + k * kT, v[k], r.x, r.y, r.z, prev_y);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[i % slices]);
            }
            if (!more) break;
            prev = slices == 1 ? -1 : row;
            prev_y = static_cast<int>(y_now);
        }
    }
    __syncwarp();
    if (*w.abort) __nanosleep(20000);   // messages that no peer waits for any more land, too
    cluster_sync();   // no CTA leaves while a peer may still write to it
    // the cluster that finishes last (a ticket in the workspace, which it takes back to zero) adds the rows' losses, or forms
    // the pairs'
    if constexpr (!kPolicy)
        if (!p.fused) return;
    if (rank != 0) return;
    __shared__ bool last;
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(p.ticket, 1u) == static_cast<uint32_t>(step) - 1u;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    if constexpr (kPolicy) block_sum<kLongThreads>(p.row_loss, in.rows, p.scale, p.loss);
    else pairs_by_warps(p, kLongThreads / 32);
    if (threadIdx.x == 0) *p.ticket = 0u;
}

// Margins, losses and the rows' coefficients: a CTA a pair.
//   margin = sum_chosen (logp - ref) - sum_rejected (logp - ref),  h = beta margin
//   loss = -(1 - e) log sigmoid(h) - e log sigmoid(-h),  d loss / d h = e sigmoid(h) - (1 - e) sigmoid(-h)
// The last CTA to finish (a ticket in the workspace, which it takes back to zero) adds the pairs' losses, in their order.
// Measured with 16 pairs of 512 rows: one CTA with a warp a pair takes 23 us.
constexpr int kPairThreads = 256;

__device__ __forceinline__ double cta_sum(double x, double* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    double s = 0.0;
    for (int w = 0; w < kPairThreads / 32; ++w) s += part[w];
    __syncthreads();
    return s;
}

template <int N>
__global__ void __launch_bounds__(kPairThreads) loss_pairs_kernel(const __grid_constant__ PrefParams p,
                                                                  const __grid_constant__ PrefPairs<N> pairs) {
    __shared__ double part[kPairThreads / 32];
    __shared__ bool last;
    pdl_wait();
    pdl_trigger();
    if (p.n_pairs == 0) {
        if (threadIdx.x == 0) *p.loss = 0.f;
        return;
    }
    const PairRows pr{pairs.p[blockIdx.x]};
    const double sum = cta_sum(margin_part(p, pr, threadIdx.x, kPairThreads), part);
    const float2 lg = pair_loss(p, sum);
    write_coefs(p, pr, lg.y, threadIdx.x, kPairThreads);
    if (threadIdx.x == 0) {
        p.margin[blockIdx.x] = static_cast<float>(sum);
        p.pair_loss[blockIdx.x] = lg.x;
        __threadfence();
        last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    double total = 0.0;
    for (int i = threadIdx.x; i < p.n_pairs; i += kPairThreads) total += static_cast<double>(__ldcg(p.pair_loss + i));
    total = cta_sum(total, part);
    if (threadIdx.x == 0) {
        *p.loss = static_cast<float>(total * static_cast<double>(p.scale));
        *p.ticket = 0u;
    }
}

constexpr int kGradVecs = 4;

// The gradient from the rows' statistics and coefficients.  Rows in falling order: the last ones the statistics pass
// read may still lie in L2.
template <typename T>
__global__ void __launch_bounds__(kT) loss_grad_kernel(const __grid_constant__ PrefParams p, int32_t chunks) {
    pdl_wait();
    pdl_trigger();
    const int64_t back = blockIdx.x / chunks;
    const int chunk = static_cast<int>(blockIdx.x - back * chunks);
    const int64_t row = p.in.rows - 1 - back;
    const RowView<T> rv(p.in, row);
    const float c = p.coef[row];
    const int begin = chunk * kGradVecs * kT + threadIdx.x;
    if (c == 0.f) {
#pragma unroll
        for (int k = 0; k < kGradVecs; ++k)
            if (begin + k * kT < rv.vecs) zero_vec(rv, begin + k * kT);
        return;
    }
    const LossRow st = p.row[row];
    const int y = static_cast<int>(p.in.labels[row]);
    uint4 v[kGradVecs];
#pragma unroll
    for (int k = 0; k < kGradVecs; ++k) v[k] = begin + k * kT < rv.vecs ? rv.load(begin + k * kT) : no_vec<T>();
#pragma unroll
    for (int k = 0; k < kGradVecs; ++k)
        if (begin + k * kT < rv.vecs) grad_vec(rv, begin + k * kT, v[k], st.top, st.inv, c, y);
}

__global__ void __launch_bounds__(1024) loss_sum_kernel(const float* x, int64_t n, float scale, float* out) {
    pdl_wait();
    pdl_trigger();
    block_sum<1024>(x, n, scale, out);
}

// Rows of at most this many vectors take the register kernel: four a thread.
constexpr int kShortVecs = 4 * kT;

template <typename T, int NV, bool kPolicy, typename P>
cudaError_t run_short(const P& p, cudaStream_t stream) {
    return launch_pdl(loss_rows_kernel<T, NV, kPolicy, P>, dim3(static_cast<unsigned>(p.in.rows)), dim3(kT), 0, stream, p);
}

// CTAs a row: as few as leave room for three slices in the ring; more while a batch of few rows leaves SMs without
// one and a slice keeps 8 KB.
int cluster_of(int64_t row_bytes, int64_t rows, int sms) {
    int c = 1;
    while (c < kMaxCluster && row_bytes > static_cast<int64_t>(c) * (kRingBytes / 3)) c *= 2;
    while (c < kMaxCluster && rows * c < sms && row_bytes >= 2 * c * 8192) c *= 2;
    return c;
}

template <typename T, bool kPolicy, typename P>
cudaError_t run_long(const P& p, int64_t vecs, int sms, cudaStream_t stream) {
    const int c = cluster_of(vecs * 16, p.in.rows, sms);
    const int slice = static_cast<int>(((vecs + c - 1) / c * 16 + 127) / 128 * 128);
    const int slices = static_cast<int>(std::min<size_t>(kMaxSlices, kRingBytes / slice));
    if (slices < 1) return cudaErrorInvalidValue;
    // clusters that fit the device at a time; the pipeline waits on nothing outside its cluster, so more would only queue
    static std::atomic<int> fits[64][4];   // of each device
    int dev = 0;
    const cudaError_t d = cudaGetDevice(&dev);
    if (d != cudaSuccess) return d;
    std::atomic<int>& fit = fits[dev & 63][c == 1 ? 0 : c == 2 ? 1 : c == 4 ? 2 : 3];
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kLongThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(slice) * slices;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(c);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    auto kernel = loss_long_rows_kernel<T, kPolicy, P>;
    int n = fit.load(std::memory_order_relaxed);
    if (n == 0) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRingBytes));
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(static_cast<unsigned>(sms / c * c));
        cfg.numAttrs = 1;
        cfg.dynamicSmemBytes = kRingBytes;   // one CTA an SM, whatever a later call's ring needs
        e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        fit.store(n, std::memory_order_relaxed);
        cfg.dynamicSmemBytes = static_cast<size_t>(slice) * slices;
    }
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(p.in.rows, n) * c));
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p, static_cast<int32_t>(c), static_cast<int32_t>(slices), static_cast<int32_t>(slice));
}

// Vectors of the longest row, however it lies.
template <typename T, typename P>
int64_t row_vecs(const P& p) {
    return (p.in.vocab + 2 * (Vec<T>::n - 1)) / Vec<T>::n;
}

template <typename T, bool kPolicy, typename P>
cudaError_t run_short(const P& p, int64_t vecs, cudaStream_t stream) {
    if (vecs <= kT) return run_short<T, 1, kPolicy>(p, stream);
    if (vecs <= 2 * kT) return run_short<T, 2, kPolicy>(p, stream);
    return run_short<T, 4, kPolicy>(p, stream);
}

template <typename T>
cudaError_t stats(const PrefParams& p, const PrefPairs<kLossMaxPairs>& pairs, int sms, bool* paired, cudaStream_t stream) {
    const int64_t vecs = row_vecs<T>(p);
    if (vecs <= kShortVecs) return run_short<T, false>(p, vecs, stream);
    PrefLong l;
    static_cast<PrefParams&>(l) = p;
    // One launch less, but each pair is one warp's work, after the last row: it goes by the longest pair and by pairs a warp.  us of
    // the statistics and the pairs' losses, fused and by a CTA a pair, rows of 32000 logits: 4 pairs of 20, 80, 128, 256, 512
    // rows 15, 21, 23, 31, 48 and 19, 23, 26, 31, 44; one of 128, 512, 4096 17, 29, 128 and 19, 26, 78; 16 of 128 44 and 44;
    // 64 of 8 29 and 25
    int32_t longest = 0;
    for (int i = 0; i < p.n_pairs; ++i) longest = std::max(longest, pairs.p[i].chosen_rows + pairs.p[i].rejected_rows);
    l.fused = p.n_pairs <= kFusedPairs && longest <= kFusedPairRows;
    if (l.fused) std::copy(pairs.p, pairs.p + p.n_pairs, l.pairs.p);
    *paired = l.fused != 0;
    return run_long<T, false>(l, vecs, sms, stream);
}

template <typename T>
cudaError_t policy_rows(const PolicyParams& p, int sms, bool* summed, cudaStream_t stream) {
    const int64_t vecs = row_vecs<T>(p);
    *summed = vecs > kShortVecs;
    return *summed ? run_long<T, true>(p, vecs, sms, stream) : run_short<T, true>(p, vecs, stream);
}

}  // namespace

cudaError_t launch_loss_stats(const PrefParams& p, const PrefPairs<kLossMaxPairs>& pairs, int sms, bool* paired, cudaStream_t stream) {
    *paired = false;
    return p.in.f32 ? stats<float>(p, pairs, sms, paired, stream) : stats<uint16_t>(p, pairs, sms, paired, stream);
}

cudaError_t launch_policy_rows(const PolicyParams& p, int sms, bool* summed, cudaStream_t stream) {
    return p.in.f32 ? policy_rows<float>(p, sms, summed, stream) : policy_rows<uint16_t>(p, sms, summed, stream);
}

cudaError_t launch_loss_pairs(const PrefParams& p, const PrefPairs<kLossMaxPairs>& pairs, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(std::max(p.n_pairs, 1)));
    if (p.n_pairs <= kFewPairs)
        return launch_pdl(loss_pairs_kernel<kFewPairs>, grid, dim3(kPairThreads), 0, stream, p,
                          reinterpret_cast<const PrefPairs<kFewPairs>&>(pairs));
    return launch_pdl(loss_pairs_kernel<kLossMaxPairs>, grid, dim3(kPairThreads), 0, stream, p, pairs);
}

cudaError_t launch_loss_grad(const PrefParams& p, cudaStream_t stream) {
    const int n = p.in.f32 ? 4 : 8;
    const int vecs = (p.in.vocab + 2 * (n - 1)) / n;
    const int32_t chunks = (vecs + kGradVecs * kT - 1) / (kGradVecs * kT);
    const dim3 grid(static_cast<unsigned>(p.in.rows * chunks));
    return p.in.f32 ? launch_pdl(loss_grad_kernel<float>, grid, dim3(kT), 0, stream, p, chunks)
                    : launch_pdl(loss_grad_kernel<uint16_t>, grid, dim3(kT), 0, stream, p, chunks);
}

cudaError_t launch_loss_sum(const float* x, int64_t n, float scale, float* out, cudaStream_t stream) {
    return launch_pdl(loss_sum_kernel, dim3(1), dim3(1024), 0, stream, x, n, scale, out);
}

}  // namespace lora
