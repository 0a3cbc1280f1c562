// The backward of the norms around a block (norm.cuh has the mathematics and the common parts).
#pragma once

#include "norm.cuh"

namespace lora {

namespace {

template <int T, int V, bool kF32, bool kSums, bool kRagged, bool kCodes>
__global__ void __launch_bounds__(T * rows_of(T), per_sm(T)) norm_bwd_kernel(const __grid_constant__ NormBwd p) {
    constexpr int R = rows_of(T);
    constexpr bool kKept = kept<T, V>();
    extern __shared__ __align__(16) uint8_t ring_memory[];
    __shared__ float shared[R][2 * 4 * (T / 32)];
    const NormShape& s = p.s;
    const int t = threadIdx.x % T, sub = threadIdx.x / T;
    const int row0 = blockIdx.x * R + sub, step = gridDim.x * R;
    const bool has_y = p.y || (kCodes && p.y8.codes);
    uint8_t* const ring = ring_memory + sub * p.stages * p.stage_bytes;
    const NormAct8 none{nullptr, nullptr};
    const Mat<T, V, kF32, kRagged, kCodes> H(p.h, p.h_ld, p.h8, s, p.at_h, t);
    const Mat<T, V, kF32, kRagged, false> Dh(p.dh, p.dh_ld, none, s, p.at_dh, t);
    const Mat<T, V, false, kRagged, false> Dx(p.dx, p.dx_ld, none, s, p.at_dx, t);
    const Mat<T, V, false, kRagged, kCodes> Y(p.y, p.y_ld, p.y8, s, p.at_y, t);
    pdl_wait();
    pdl_trigger();
    const int mine = kRagged ? units_of<T, V>(t, s.width) : V;
    const auto fetch = [&](int row, int slot) {
        if (row < s.rows) {
            uint8_t* const a = ring + slot * p.stage_bytes;
            Dx.fetch(a, row, t, s.width);
            H.fetch(a, row, t, s.width);
            Dh.fetch(a, row, t, s.width);
            Y.fetch(a, row, t, s.width);
        }
        copies_end();
    };
    for (int i = 0; i < p.stages; ++i) {
        uint8_t* const a = ring + i * p.stage_bytes;
        if (s.w.p) {
            H.clear(a);
            Dx.clear(a);
        }
        Dh.clear(a);
        if (has_y) Y.clear(a);
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
    F2 sum_w[kSums ? V : 1][4], sum_k[kSums ? V : 1][4];
    if (kSums) {
#pragma unroll
        for (int i = 0; i < (kSums ? V : 1); ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) sum_w[i][k] = sum_k[i][k] = both(0.f);
    }
    const auto gate_of = [&](int row) { return s.row_gate.p && row < s.rows ? one_weight(s.row_gate, row) : 1.f; };
    float rg = 1.f, next_rg = gate_of(row0);   // of the row that z is of, and of the one after
    F2 d[V][4];             // the gradient of the stream, then z
    float inverse_y = 1.f;  // of the row that z is of: 1 / rms(y)
    // q[1], q[2], q[3]: sums of h^2, t h, y^2
    const auto squares = [&](int row, uint8_t* stage, float (&q)[4]) {
        F2 hh = both(0.f), th = both(0.f), yy = both(0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (kRagged && i >= mine) break;
            if (s.w.p) {
                F2 h[4], dx[4], f[4];
                H.template read<kKeep>(h, stage, row, i, t);
                Dx.template read<kKeep>(dx, stage, row, i, t);
                if (!kKept) main_factors<T>(f, s, i, t);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    hh = fma2(h[k], h[k], hh);
                    th = fma2(h[k], mul(dx[k], kKept ? fw[kKept ? i : 0][k] : f[k]), th);
                }
            }
            if (s.post.p) {
                F2 y[4];
                Y.template read<kKeep>(y, stage, row, i, t);
#pragma unroll
                for (int k = 0; k < 4; ++k) yy = fma2(y[k], y[k], yy);
            }
        }
        q[1] = total(hh);
        q[2] = total(th);
        q[3] = total(yy);
    };
    // From these sums: the stream's gradient of a row, stored, then z; returns the sum of z v.
    const auto stream = [&](int row, uint8_t* stage, const float (&q)[4]) {
        float r = inverse_rms(q[1], s), m = q[2] * r;
        inverse_y = s.post.p ? inverse_rms(q[3], s) : 1.f;
        if (too_large(q[1]) || too_large(q[3])) {
            float f[4] = {0.f, 0.f, 0.f, 0.f};
            if (s.w.p) {
                const bool codes = kCodes && p.h8.codes;
                const RowAt<kF32> at{codes ? p.h8.codes + static_cast<uint64_t>(s.codes_ld) * static_cast<uint32_t>(row) : static_cast<const uint8_t*>(p.h) + static_cast<uint64_t>(p.h_ld) * static_cast<uint32_t>(row),
                                     codes ? p.h8.scales + static_cast<uint64_t>(s.scales_ld) * static_cast<uint32_t>(row) : nullptr};
                const uint16_t* dx = reinterpret_cast<const uint16_t*>(reinterpret_cast<const uint8_t*>(p.dx) + static_cast<uint64_t>(p.dx_ld) * static_cast<uint32_t>(row));
                const float2 a = small_sums(at, dx, s.w, s.offset, t, T, s.width);
                f[1] = a.x;
                f[2] = a.y;
            }
            if (s.post.p) {
                const bool codes = kCodes && p.y8.codes;
                const RowAt<false> at{codes ? p.y8.codes + static_cast<uint64_t>(s.codes_ld) * static_cast<uint32_t>(row) : reinterpret_cast<const uint8_t*>(p.y) + static_cast<uint64_t>(p.y_ld) * static_cast<uint32_t>(row),
                                      codes ? p.y8.scales + static_cast<uint64_t>(s.scales_ld) * static_cast<uint32_t>(row) : nullptr};
                f[3] = small_sums(at, nullptr, s.w, 0.f, t, T, s.width).x;
            }
            sums.add(f);
            if (too_large(q[1])) {
                r = inverse_rms_small(f[1], s);
                m = f[2] * r;
                r *= kSmall;
            }
            if (s.post.p && too_large(q[3])) inverse_y = inverse_rms_small(f[3], s) * kSmall;
        }
        m *= s.inv_width;
        rg = next_rg;
        next_rg = gate_of(row + step);
        F2 along = both(0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (kRagged && i >= mine) break;
            Dh.template read<kOnce>(d[i], stage, row, i, t);
            if (s.w.p) {
                F2 h[4], dx[4], f[4];
                H.template read<kPlain>(h, stage, row, i, t);
                Dx.template read<kPlain>(dx, stage, row, i, t);
                if (!kKept) main_factors<T>(f, s, i, t);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const F2 n = mul(h[k], both(r));
                    if (kSums) sum_w[kSums ? i : 0][k] = fma2(dx[k], n, sum_w[kSums ? i : 0][k]);
                    d[i][k] = fma2(fma2(n, both(-m), mul(dx[k], kKept ? fw[kKept ? i : 0][k] : f[k])), both(r), d[i][k]);
                }
            }
            Unit<kF32> out;
            out.put(d[i]);
            store_unit<T, kF32, kRagged>(out, static_cast<uint8_t*>(p.dh_out) + static_cast<uint64_t>(p.dh_out_ld) * static_cast<uint32_t>(row), i, t, s.width);
            if (!has_y) continue;
            F2 y[4], f[4];
            if (kRagged && !s.post.p) Y.template read<kOnce>(y, stage, row, i, t);
            else Y.template read<kPlain>(y, stage, row, i, t);
            if (!kKept) block_factors<T>(f, s, i, t);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const F2 v = mul(y[k], both(inverse_y));
                if (kSums) sum_k[kSums ? i : 0][k] = fma2(mul(d[i][k], both(rg)), v, sum_k[kSums ? i : 0][k]);
                d[i][k] = mul(d[i][k], kKept ? fc[kKept ? i : 0][k] : f[k]);
                along = fma2(d[i][k], v, along);
            }
        }
        return total(along);
    };
    // dy and the row gate's gradient of the row whose z is held
    const auto block = [&](int row, uint8_t* stage, float along) {
        if (!has_y) return;
        if (p.drow && t == 0) p.drow[row] = along;
        if (!p.dy) return;
        const float m = s.post.p ? along * rg * s.inv_width : 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (kRagged && i >= mine) break;
            F2 f[4];
            if (s.post.p) {
                F2 y[4];
                Y.template read<kPlain>(y, stage, row, i, t);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    f[k] = mul(fma2(mul(y[k], both(inverse_y)), both(-m), mul(d[i][k], both(rg))), both(inverse_y));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) f[k] = mul(d[i][k], both(rg));
            }
            Unit<false> out;
            out.put(f);
            store_unit<T, false, kRagged>(out, reinterpret_cast<uint8_t*>(p.dy) + static_cast<uint64_t>(p.dy_ld) * static_cast<uint32_t>(row), i, t, s.width);
        }
    };
    const bool second = s.post.p || p.drow;   // the sum of z v is needed
    if (!kKept) {   // wide rows: one at a time
        for (int row = row0; row < s.rows; row += step) {
            fetch(row, 0);
            copies_wait(0);
            float q[4] = {0.f, 0.f, 0.f, 0.f};
            squares(row, ring, q);
            sums.add(q);
            q[0] = stream(row, ring, q);
            if (second) sums.add(q);
            block(row, ring, q[0]);
        }
    } else {
        int slot = -1;
        float now_sums[4] = {0.f, 0.f, 0.f, 0.f};   // of the row in `slot`
        for (int row = row0 - step;; row += step) {
            const bool now = slot >= 0, more = row + step < s.rows;
            const int after = slot + 1 == p.stages ? 0 : slot + 1;
            float q[4] = {0.f, 0.f, 0.f, 0.f};   // this row's z v; the next row's h^2, t h, y^2
            if (now) {
                fetch(row + (p.stages - 1) * step, slot == 0 ? p.stages - 1 : slot - 1);
                q[0] = stream(row, ring + slot * p.stage_bytes, now_sums);
            }
            if (more) {
                copies_wait(p.stages - 2);
                squares(row + step, ring + after * p.stage_bytes, q);
            }
            if (more || (now && second)) sums.add(q);
            if (now) block(row, ring + slot * p.stage_bytes, q[0]);
            if (!more) break;
#pragma unroll
            for (int k = 0; k < 4; ++k) now_sums[k] = q[k];
            slot = after;
        }
    }
    if (kSums) {
        // the CTA's rows are added first, in a fixed order, through the ring's memory
        float* gathered = reinterpret_cast<float*>(ring_memory);
        constexpr int kOne = 2 * T * V * 8;
        if (R > 1) {
            __syncthreads();
            if (sub > 0) {
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        F2* to = reinterpret_cast<F2*>(gathered + (sub - 1) * kOne);
                        to[((i * 4 + k) * 2) * T + t] = sum_w[kSums ? i : 0][k];
                        to[((i * 4 + k) * 2 + 1) * T + t] = sum_k[kSums ? i : 0][k];
                    }
            }
            __syncthreads();
            if (sub > 0) return;
            for (int j = 0; j < R - 1; ++j) {
                const F2* from = reinterpret_cast<const F2*>(gathered + j * kOne);
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        sum_w[kSums ? i : 0][k] = add2(sum_w[kSums ? i : 0][k], from[((i * 4 + k) * 2) * T + t]);
                        sum_k[kSums ? i : 0][k] = add2(sum_k[kSums ? i : 0][k], from[((i * 4 + k) * 2 + 1) * T + t]);
                    }
            }
        }
        float* part = p.part + static_cast<int64_t>(blockIdx.x) * 2 * s.width;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int c = (i * T + t) * 8 + 2 * k;
                const float2 a = parts(sum_w[kSums ? i : 0][k]), b = parts(sum_k[kSums ? i : 0][k]);
                if (c < s.width) part[c] = a.x, part[s.width + c] = b.x;
                if (c + 1 < s.width) part[c + 1] = a.y, part[s.width + c + 1] = b.y;
            }
    }
}

template <bool kSums, bool kCodes>
cudaError_t launch_norm_bwd_form(NormBwd& p, int sms, cudaStream_t stream) {
    return by_width(p.s.width, p.s.ragged, [&](auto t, auto v, auto r) {
        constexpr int T = decltype(t)::value, V = decltype(v)::value, R = rows_of(T);
        constexpr bool K = decltype(r)::value;
        const int wide = stage_bytes_of(T, V, p.s.f32 ? 4 : 2, K), half = stage_bytes_of(T, V, 2, K), codes = T * V * 12;
        uint32_t at = 0;
        const auto place = [&at](bool there, int bytes) {
            const uint32_t was = at;
            if (there) at += bytes;
            return was;
        };
        p.at_dx = place(p.dx, half);
        p.at_h = place(p.h || p.h8.codes, p.h8.codes ? codes : wide);
        p.at_dh = place(true, wide);
        p.at_y = place(p.y || p.y8.codes, p.y8.codes ? codes : half);
        p.stage_bytes = at;
        const RingPlan plan = ring_plan(R * p.stage_bytes, per_sm(T), kept<T, V>());
        p.stages = plan.stages;
        const int grid = std::min((p.s.rows + R - 1) / R, sms * plan.per_sm);
        p.groups = grid;
        auto* k = p.s.f32 ? norm_bwd_kernel<T, V, true, kSums, K, kCodes> : norm_bwd_kernel<T, V, false, kSums, K, kCodes>;
        // the rows' rings, in whose place the CTA's sums are gathered at the end
        const int memory = std::max<int>(R * p.stages * p.stage_bytes, kSums ? (R - 1) * 2 * T * V * 8 * 4 : 0);
        static std::atomic<uint64_t> ready[2];   // of this form, by the stream's type
        const cudaError_t e = let_rings(k, ready[p.s.f32 ? 1 : 0]);
        return e != cudaSuccess ? e : launch_pdl(k, dim3(grid), dim3(T * R), memory, stream, p);
    });
}

}  // namespace

}  // namespace lora
