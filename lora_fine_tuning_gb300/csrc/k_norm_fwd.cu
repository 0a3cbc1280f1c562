// The forward of the norms around a block (norm.cuh has the mathematics and the common parts).
#include "norm.cuh"

namespace lora {

namespace {

template <int T, int V, bool kF32, bool kRagged>
__global__ void __launch_bounds__(T * rows_of(T), per_sm(T)) norm_fwd_kernel(const __grid_constant__ NormFwd p) {
    constexpr int R = rows_of(T);
    constexpr bool kKept = kept<T, V>();
    extern __shared__ __align__(16) uint8_t ring_memory[];
    __shared__ float shared[R][2 * 4 * (T / 32)];
    const NormShape& s = p.s;
    const int t = threadIdx.x % T, sub = threadIdx.x / T;
    uint8_t* const ring = ring_memory + sub * p.stages * p.stage_bytes;
    const NormAct8 none{nullptr, nullptr};
    const Mat<T, V, kF32, kRagged, false> H(p.h, p.h_ld, none, s, 0, t);
    const Mat<T, V, false, kRagged, false> Y(p.y, p.y_ld, none, s, p.at_y, t);
    pdl_wait();
    pdl_trigger();
    const int mine = kRagged ? units_of<T, V>(t, s.width) : V;
    const int step = gridDim.x * R, row0 = blockIdx.x * R + sub;
    const auto fetch = [&](int row, int slot) {
        if (row < s.rows) {
            H.fetch(ring + slot * p.stage_bytes, row, t, s.width);
            Y.fetch(ring + slot * p.stage_bytes, row, t, s.width);
        }
        copies_end();
    };
    for (int i = 0; i < p.stages; ++i) {
        H.clear(ring + i * p.stage_bytes);
        if (p.y) Y.clear(ring + i * p.stage_bytes);
    }
    for (int i = 0; i + 1 < p.stages; ++i) fetch(row0 + i * step, i);
    F2 fw[kKept ? V : 1][4], fc[kKept ? V : 1][4];
    if (kKept) {
#pragma unroll
        for (int i = 0; i < (kKept ? V : 1); ++i) {
            main_factors<T>(fw[i], s, i, t);
            block_factors<T>(fc[i], s, i, t);
        }
    }
    RowSums<T> sums(shared[sub], 1 + sub);
    const auto gate_of = [&](int row) { return s.row_gate.p && row < s.rows ? one_weight(s.row_gate, row) : 1.f; };
    float gate = gate_of(row0);
    F2 h[V][4];
    // the sum of y^2
    const auto block_squares = [&](int row, uint8_t* stage) {
        F2 q = both(0.f);
        if (s.post.p) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (kRagged && i >= mine) break;
                F2 y[4];
                Y.template read<kKeep>(y, stage, row, i, t);
#pragma unroll
                for (int k = 0; k < 4; ++k) q = fma2(y[k], y[k], q);
            }
        }
        return total(q);
    };
    // h' of a row, stored; the sum of its squares
    const auto join = [&](int row, uint8_t* stage, float squares) {
        float c = gate;
        if (p.y) {
            gate = gate_of(row + step);   // on its way before the next row needs it
            if (s.post.p) {
                float r = inverse_rms(squares, s);
                if (too_large(squares)) {
                    const RowAt<false> at{reinterpret_cast<const uint8_t*>(p.y) + static_cast<uint64_t>(p.y_ld) * static_cast<uint32_t>(row), nullptr};
                    float q[4] = {small_sums(at, nullptr, s.w, 0.f, t, T, s.width).x, 0.f, 0.f, 0.f};
                    sums.add(q);
                    r = inverse_rms_small(q[0], s) * kSmall;
                }
                c *= r;
            }
        }
        F2 q = both(0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (kRagged && i >= mine) break;
            H.template read<kOnce>(h[i], stage, row, i, t);
            if (p.y) {
                F2 y[4], f[4];
                if (kRagged && !s.post.p) Y.template read<kOnce>(y, stage, row, i, t);
                else Y.template read<kPlain>(y, stage, row, i, t);
                if (!kKept) block_factors<T>(f, s, i, t);
                if (p.y8.codes) {
                    Unit<false> u;
                    u.put(y);
                    store_act8<T>(u, p.y8, s, row, i, t);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) h[i][k] = fma2(mul(y[k], both(c)), kKept ? fc[kKept ? i : 0][k] : f[k], h[i][k]);
                Unit<kF32> out;
                out.put(h[i]);
                store_unit<T, kF32, kRagged>(out, static_cast<uint8_t*>(p.h_out) + static_cast<uint64_t>(p.h_out_ld) * static_cast<uint32_t>(row), i, t, s.width);
            }
            if (p.h8.codes) {
                Unit<false> u;
                u.put(h[i]);
                store_act8<T>(u, p.h8, s, row, i, t);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) q = fma2(h[i][k], h[i][k], q);
        }
        return total(q);
    };
    // x of the row whose h' is held
    const auto norm = [&](int row, float squares) {
        if (!s.w.p) return;
        float r = inverse_rms(squares, s);
        if (too_large(squares)) {
            F2 a = both(0.f);
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) if (!kRagged || i < mine) a = fma2(mul(h[i][k], both(kSmall)), mul(h[i][k], both(kSmall)), a);
            float q[4] = {total(a), 0.f, 0.f, 0.f};
            sums.add(q);
            r = inverse_rms_small(q[0], s) * kSmall;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (kRagged && i >= mine) break;
            F2 f[4];
            if (!kKept) main_factors<T>(f, s, i, t);
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = mul(mul(h[i][k], both(r)), kKept ? fw[kKept ? i : 0][k] : f[k]);
            Unit<false> x;
            x.put(f);
            if (p.x) store_unit<T, false, kRagged>(x, reinterpret_cast<uint8_t*>(p.x) + static_cast<uint64_t>(p.x_ld) * static_cast<uint32_t>(row), i, t, s.width);
            if (p.x8.codes) store_act8<T>(x, p.x8, s, row, i, t);
        }
    };
    if (!kKept) {   // wide rows: one at a time
        for (int row = row0; row < s.rows; row += step) {
            fetch(row, 0);
            copies_wait(0);
            float q[4] = {0.f, block_squares(row, ring), 0.f, 0.f};
            if (s.post.p) sums.add(q);
            q[0] = join(row, ring, q[1]);
            if (s.w.p) sums.add(q);
            norm(row, q[0]);
        }
        return;
    }
    int slot = -1;
    float block_sum = 0.f;   // of y^2, of the row in `slot`
    for (int row = row0 - step;; row += step) {
        const bool now = slot >= 0, more = row + step < s.rows;
        const int after = slot + 1 == p.stages ? 0 : slot + 1;
        float q[4] = {0.f, 0.f, 0.f, 0.f};   // sums of this row's h'^2 and of the next row's y^2
        if (now) {
            fetch(row + (p.stages - 1) * step, slot == 0 ? p.stages - 1 : slot - 1);
            q[0] = join(row, ring + slot * p.stage_bytes, block_sum);
        }
        if (more) {
            copies_wait(p.stages - 2);
            q[1] = block_squares(row + step, ring + after * p.stage_bytes);
        }
        if (s.post.p || (now && s.w.p)) sums.add(q);
        if (now) norm(row, q[0]);
        if (!more) return;
        block_sum = q[1];
        slot = after;
    }
}

}  // namespace

cudaError_t launch_norm_fwd(const NormFwd& given, int sms, cudaStream_t stream) {
    return by_width(given.s.width, given.s.ragged, [&](auto t, auto v, auto r) {
        constexpr int T = decltype(t)::value, V = decltype(v)::value, R = rows_of(T);
        constexpr bool K = decltype(r)::value;
        NormFwd p = given;
        p.at_y = stage_bytes_of(T, V, p.s.f32 ? 4 : 2, K);
        p.stage_bytes = p.at_y + (p.y ? stage_bytes_of(T, V, 2, K) : 0);
        const RingPlan plan = ring_plan(R * p.stage_bytes, per_sm(T), kept<T, V>());
        p.stages = plan.stages;
        const int grid = std::min((p.s.rows + R - 1) / R, sms * plan.per_sm);
        auto* k = p.s.f32 ? norm_fwd_kernel<T, V, true, K> : norm_fwd_kernel<T, V, false, K>;
        static std::atomic<uint64_t> ready[2];   // of this form, by the stream's type
        const cudaError_t e = let_rings(k, ready[p.s.f32 ? 1 : 0]);
        return e != cudaSuccess ? e : launch_pdl(k, dim3(grid), dim3(T * R), R * p.stages * p.stage_bytes, stream, p);
    });
}

}  // namespace lora
