// Losses on logits, forward and gradient.
//
//   logp_t = z_ty - max - log sum_v exp(z_tv - max),   d loss / d z_tv = c_t (1[v = y_t] - p_tv),   c_t = d loss / d logp_t
//
// Both losses are bound by the logits: read once, and the gradient written once.  The policy loss depends on one row
// at a time, so a row stays in the registers of the CTAs of a cluster from its one read to the write of its gradient.
// The preference loss needs the sums over both responses of a pair before any gradient: a pass over the logits for the
// statistics, the pairs' losses in one CTA, and a pass that reads the logits again and writes the gradient.
//
// All statistics are fp32 relative to the row's maximum (p of the label is then exact to 2^-23 also near 1, where
// 1 - p is the gradient); sums over tokens are fp64 in a fixed order.

#include "attn.cuh"
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
    static __device__ __forceinline__ void get(uint4 v, float (&x)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                          pack_bf16x2(x[6], x[7]));
    }
    static __device__ __forceinline__ float one(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
    static __device__ __forceinline__ uint16_t bits(float x) { return bf16_bits(x); }
};
template <>
struct Vec<float> {
    static constexpr int n = 4;
    static constexpr uint32_t kFill = 0xFF800000u;
    static __device__ __forceinline__ void get(uint4 v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
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
        float x[Vec<T>::n];
#pragma unroll
        for (int j = 0; j < Vec<T>::n; ++j) x[j] = e + j >= 0 && e + j < vocab ? Vec<T>::one(z + e + j) : neg_inf();
        return Vec<T>::put(x);
    }
    __device__ __forceinline__ void store(int i, const float (&x)[Vec<T>::n]) const {
        const int e = i * Vec<T>::n - skew;
        if (same && whole(i)) {
            __stcs(reinterpret_cast<uint4*>(dz + e), Vec<T>::put(x));
            return;
        }
#pragma unroll
        for (int j = 0; j < Vec<T>::n; ++j)
            if (e + j >= 0 && e + j < vocab) dz[e + j] = Vec<T>::bits(x[j]);
    }
};

// exp(x - top); 0 for x = -inf whatever top is.
__device__ __forceinline__ float exp_from(float x, float top) { return ex2((x - top) * kLog2e); }

// Joins two (maximum, sum) pairs.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
    const float t = fmaxf(m, m2);
    const float a = m == t ? s : s * exp_from(m, t);
    const float b = m2 == t ? s2 : s2 * exp_from(m2, t);
    m = t;
    s = a + b;
}

// c (1[v = y] - p) of one vector.
template <typename T>
__device__ __forceinline__ void grad_vec(const RowView<T>& rv, int i, uint4 raw, float top, float inv, float c, int y) {
    constexpr int n = Vec<T>::n;
    float x[n];
    Vec<T>::get(raw, x);
    const int at = y - (i * n - rv.skew);
    const float f = -c * inv;
#pragma unroll
    for (int j = 0; j < n; ++j) x[j] = f * exp_from(x[j], top);
    if (static_cast<unsigned>(at) < static_cast<unsigned>(n)) {
#pragma unroll
        for (int j = 0; j < n; ++j)
            if (j == at) x[j] += c;
    }
    rv.store(i, x);
}

template <typename T>
__device__ __forceinline__ void zero_vec(const RowView<T>& rv, int i) {
    float x[Vec<T>::n];
#pragma unroll
    for (int j = 0; j < Vec<T>::n; ++j) x[j] = 0.f;
    rv.store(i, x);
}

// What the policy loss makes of a row's logp: its loss, and c = d loss / d logp (both without `scale`).
__device__ __forceinline__ void policy_row(const PolicyParams& p, int64_t row, float logp, float* loss, float* c) {
    const float a = p.adv[row];
    const float r = expf(logp - p.old_logp[row]);
    const float ra = r * a;
    const float clipped = fminf(fmaxf(r, p.lo), p.hi) * a;
    const bool free = a >= 0.f ? r <= p.hi : r >= p.lo;
    float l = -fminf(ra, clipped), g = free ? -ra : 0.f;
    if (ra != ra) l = g = ra;   // fminf would drop a NaN
    if (p.ref) {
        const float x = p.ref[row] - logp, e = expm1f(x);
        l += p.kl * (e - x);
        g -= p.kl * e;
    }
    *loss = l;
    *c = g;
}

// A row's statistics from the registers of one cluster: NV vectors a thread.  kPolicy: the whole policy loss of the
// row, gradient included; else the statistics for the preference loss.
template <typename T, int NV, bool kPolicy, typename P>
__global__ void __launch_bounds__(kT, NV <= 8 ? 2 : 1) loss_rows_kernel(const __grid_constant__ P p, int32_t cluster) {
    __shared__ float2 part[kT / 32];
    __shared__ float2 peers[8];
    __shared__ float2 result;   // top, inv
    __shared__ float coef;
    pdl_wait();
    pdl_trigger();
    const int64_t row = blockIdx.x / cluster;
    const int rank = static_cast<int>(blockIdx.x - row * cluster);
    const LossLogits& in = p.in;
    const RowView<T> rv(in, row);
    const int per = (rv.vecs + cluster - 1) / cluster;
    const int begin = rank * per, end = min(begin + per, rv.vecs);
    const int64_t y64 = in.labels[row];
    const bool counts = y64 >= 0 && y64 < in.vocab;
    if (!counts) {   // the same in every CTA of the cluster; the row's logits are not read
        if (rank == 0 && threadIdx.x == 0) {
            in.logp[row] = 0.f;
            if constexpr (kPolicy) p.row_loss[row] = 0.f;
            else p.coef[row] = 0.f;
        }
        if (kPolicy && in.dz)
            for (int i = begin + threadIdx.x; i < end; i += kT) zero_vec(rv, i);
        return;
    }
    // a CTA's shared memory may be written by its peers once all of the cluster have started
    if (cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int y = static_cast<int>(y64);
    uint4 v[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = begin + k * kT + threadIdx.x;
        v[k] = make_uint4(Vec<T>::kFill, Vec<T>::kFill, Vec<T>::kFill, Vec<T>::kFill);
        if (i < end) v[k] = rv.load(i);
    }
    float zy = 0.f;
    if (threadIdx.x == 0) zy = Vec<T>::one(rv.z + y);
    float m = neg_inf(), s = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        float x[Vec<T>::n];
        Vec<T>::get(v[k], x);
#pragma unroll
        for (int j = 0; j < Vec<T>::n; ++j) m = fmaxf(m, x[j]);
    }
    const float mt = m == neg_inf() ? 0.f : m;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        float x[Vec<T>::n];
        Vec<T>::get(v[k], x);
#pragma unroll
        for (int j = 0; j < Vec<T>::n; ++j) s += exp_from(x[j], mt);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        join(m, s, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, s, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(m, s);
    __syncthreads();
    if (cluster > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (threadIdx.x < 32) {
        const float2 q = threadIdx.x < kT / 32 ? part[threadIdx.x] : make_float2(neg_inf(), 0.f);
        m = q.x;
        s = q.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            join(m, s, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, s, o));
        if (cluster > 1 && static_cast<int>(threadIdx.x) < cluster) {
            // this CTA's pair to every CTA of the cluster
            uint32_t remote;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(&peers[rank])), "r"(threadIdx.x));
            asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote), "f"(m), "f"(s) : "memory");
        }
    }
    if (cluster > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    if (threadIdx.x == 0) {
        if (cluster > 1) {
            m = neg_inf();
            s = 0.f;
            for (int i = 0; i < cluster; ++i) join(m, s, peers[i].x, peers[i].y);
        }
        const float logp = (zy - m) - logf(s);
        result = make_float2(m, 1.f / s);
        if constexpr (kPolicy) {
            float loss, c;
            policy_row(p, row, logp, &loss, &c);
            coef = p.scale * c;
            if (rank == 0) p.row_loss[row] = loss;
        } else {
            if (rank == 0) {
                p.row[row] = LossRow{m, 1.f / s};
                p.coef[row] = 0.f;   // rows of no pair; the pairs' rows get theirs from the pairs kernel
            }
        }
        if (rank == 0) in.logp[row] = logp;
    }
    if constexpr (kPolicy) {
        if (!in.dz) return;
        __syncthreads();
        const float top = result.x, inv = result.y, c = coef;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = begin + k * kT + threadIdx.x;
            if (i < end) grad_vec(rv, i, v[k], top, inv, c, y);
        }
    }
}

// Margins, losses and the rows' coefficients of all pairs, by one CTA: a warp a pair.
//   margin = sum_chosen (logp - ref) - sum_rejected (logp - ref),  h = beta margin
//   loss = -(1 - e) log sigmoid(h) - e log sigmoid(-h),  d loss / d h = e sigmoid(h) - (1 - e) sigmoid(-h)
template <int N>
__global__ void __launch_bounds__(1024) loss_pairs_kernel(const __grid_constant__ PrefParams p,
                                                          const __grid_constant__ PrefPairs<N> pairs) {
    __shared__ double warp_loss[32];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const auto counts = [&](int64_t r) { return p.in.labels[r] >= 0 && p.in.labels[r] < p.in.vocab; };
    double total = 0.0;
    for (int i = warp; i < p.n_pairs; i += 32) {
        const PrefPair q = pairs.p[i];
        double sum = 0.0;
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
            const int64_t from = side == 0 ? q.chosen : q.rejected;
            const int n = side == 0 ? q.chosen_rows : q.rejected_rows;
            double part = 0.0;
#pragma unroll 4
            for (int r = lane; r < n; r += 32)
                if (counts(from + r))
                    part += static_cast<double>(p.in.logp[from + r]) - (p.ref ? static_cast<double>(p.ref[from + r]) : 0.0);
            sum += side == 0 ? part : -part;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float h = static_cast<float>(static_cast<double>(p.beta) * sum);
        const float e = p.smoothing;
        // log sigmoid(h) = min(h, 0) - log1p(exp(-|h|)),  log sigmoid(-h) = log sigmoid(h) - h
        const float tail = log1pf(expf(-fabsf(h)));
        const float loss = (1.f - e) * (tail - fminf(h, 0.f)) + e * (tail + fmaxf(h, 0.f));
        const float small = expf(-fabsf(h)), s_neg = (h >= 0.f ? small : 1.f) / (1.f + small);   // sigmoid(-h)
        const float s_pos = (h >= 0.f ? 1.f : small) / (1.f + small);
        const float g = h != h ? h : p.scale * p.beta * (e * s_pos - (1.f - e) * s_neg);
        if (lane == 0) {
            p.margin[i] = static_cast<float>(sum);
            total += h != h ? h : loss;
        }
        for (int r = lane; r < q.chosen_rows; r += 32)
            if (counts(q.chosen + static_cast<int64_t>(r))) p.coef[q.chosen + static_cast<int64_t>(r)] = g;
        for (int r = lane; r < q.rejected_rows; r += 32)
            if (counts(q.rejected + static_cast<int64_t>(r))) p.coef[q.rejected + static_cast<int64_t>(r)] = -g;
    }
    if (lane == 0) warp_loss[warp] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 32; ++w) total += warp_loss[w];
        *p.loss = static_cast<float>(total * static_cast<double>(p.scale));
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
    for (int k = 0; k < kGradVecs; ++k)
        if (begin + k * kT < rv.vecs) v[k] = rv.load(begin + k * kT);
#pragma unroll
    for (int k = 0; k < kGradVecs; ++k)
        if (begin + k * kT < rv.vecs) grad_vec(rv, begin + k * kT, v[k], st.top, st.inv, c, y);
}

// out = scale * sum x, in fp64 in a fixed order, by one CTA.
__global__ void __launch_bounds__(1024) loss_sum_kernel(const float* x, int64_t n, float scale, float* out) {
    __shared__ double part[32];
    pdl_wait();
    pdl_trigger();
    double s = 0.0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < n; i += 1024) s += static_cast<double>(x[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 32; ++w) s += part[w];
        *out = static_cast<float>(s * static_cast<double>(scale));
    }
}

// CTAs a row: as few as hold it with eight vectors a thread (sixteen for the longest rows), more while a batch of few
// rows leaves SMs without one and each thread keeps a vector.
int cluster_of(int vecs, int64_t rows, int sms) {
    int c = 1;
    while (c < 8 && c * kT * 8 < vecs) c *= 2;
    while (c < 8 && rows * c < sms && vecs >= 2 * c * kT) c *= 2;
    return c;
}

template <typename T, int NV, bool kPolicy, typename P>
cudaError_t run_rows(const P& p, int cluster, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.in.rows * cluster));
    cfg.blockDim = dim3(kT);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, loss_rows_kernel<T, NV, kPolicy, P>, p, static_cast<int32_t>(cluster));
}

template <typename T, bool kPolicy, typename P>
cudaError_t rows_of(const P& p, int sms, cudaStream_t stream) {
    const int vecs = (p.in.vocab + 2 * (Vec<T>::n - 1)) / Vec<T>::n;   // of the longest row, however it lies
    const int c = cluster_of(vecs, p.in.rows, sms);
    const int each = ((vecs + c - 1) / c + kT - 1) / kT;
    if (each <= 1) return run_rows<T, 1, kPolicy>(p, c, stream);
    if (each <= 2) return run_rows<T, 2, kPolicy>(p, c, stream);
    if (each <= 4) return run_rows<T, 4, kPolicy>(p, c, stream);
    if (each <= 8) return run_rows<T, 8, kPolicy>(p, c, stream);
    if (each <= 17) return run_rows<T, 17, kPolicy>(p, c, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_loss_stats(const PrefParams& p, int sms, cudaStream_t stream) {
    return p.in.f32 ? rows_of<float, false>(p, sms, stream) : rows_of<uint16_t, false>(p, sms, stream);
}

cudaError_t launch_policy_rows(const PolicyParams& p, int sms, cudaStream_t stream) {
    return p.in.f32 ? rows_of<float, true>(p, sms, stream) : rows_of<uint16_t, true>(p, sms, stream);
}

cudaError_t launch_loss_pairs(const PrefParams& p, const PrefPairs<kLossMaxPairs>& pairs, cudaStream_t stream) {
    if (p.n_pairs <= kFewPairs)
        return launch_pdl(loss_pairs_kernel<kFewPairs>, dim3(1), dim3(1024), 0, stream, p,
                          reinterpret_cast<const PrefPairs<kFewPairs>&>(pairs));
    return launch_pdl(loss_pairs_kernel<kLossMaxPairs>, dim3(1), dim3(1024), 0, stream, p, pairs);
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
