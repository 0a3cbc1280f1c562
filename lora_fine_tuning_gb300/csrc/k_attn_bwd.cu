// Backward of causal softmax attention over packed sequences with grouped heads.
//
//   P = exp(scale Q K^T - lse),  delta_i = sum_d dO_id O_id,  dP = dO V^T,  dS = P (dP - delta)
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO,   dK and dV summed over the query heads of a group
//
// Two passes: dQ, a CTA a 128-row query tile over its keys (delta on the way); dK and dV, a CTA a 128-key tile over the
// query tiles of all heads of its group.  Each gradient element is summed by one CTA in a fixed order, in TMEM in fp32:
// the results are the same from call to call, and no partial sum goes through memory.  The price is that S and dP are
// formed twice (seven products instead of five).  dS and, for dV, P are rounded to bf16, the tensor cores' operand type;
// dS comes from P and dP in fp32.  P is formed with the approximate exponential (2^-22).
//
// delta: the dQ pass starts from the O that it is given, in bf16.  Where P gathers on few keys, dP - delta cancels, and this
// rounding of O grows: 0.006 of dQ and of dK (2-norm) for scores with a standard deviation of 12, where dS in bf16 alone gives
// 0.0024.  But P sums to 1 over a row, so the row's sum of P (dP - delta), in fp32 before any rounding, is what delta lacks.
// The dQ pass adds it up and hands the whole delta to the dK and dV pass: dK is off by 0.0024, at 3% of the dQ pass's time.
// dQ itself keeps the first delta: its correction, the missing part times P K, would take a fourth product, and TMEM has no
// room for its sums.
//
// Bound by the tensor cores on long sequences: four of 4096 tokens, 64/8 heads of 128, take 1140 us for dQ (three
// products, 880 us at the cuBLAS rate) and 1270 to 1310 us for dK and dV (four products, 1173 us).  On short ones by the start
// of a CTA, whose first tiles of 32 KB arrive together.
#include "attn.cuh"
#include "kernels.h"

namespace lora {

namespace {

constexpr int kThreads = 320;   // warps 0-7: scores and gradients of scores; warp 8: TMA; warp 9: MMAs

// The two groups of four warps share every 128 x 128 tile: group g takes columns [64 g, 64 g + 64).  A group packs
// its bf16 results into the first 32 of the TMEM columns that it read itself, so neither group waits for the other:
// K step ks (16 values, 8 columns) of the tile as an A operand starts at column (ks / 4) * 64 + (ks % 4) * 8.
__device__ __forceinline__ uint32_t a_col(int ks) { return (ks >> 2) * 64 + (ks & 3) * 8; }

// 64 columns of this thread's row.
__device__ __forceinline__ void ld64(uint32_t taddr, uint32_t (&v)[2][32]) {
    tmem_ld32(taddr, v[0]);
    tmem_ld32(taddr + 32, v[1]);
    tmem_ld_wait(v);
}

// Barrier among the T threads of the score warps.
template <int T>
__device__ __forceinline__ void score_sync() { asm volatile("bar.sync 1, %0;" ::"n"(T) : "memory"); }

// Columns 2 e and 2 e + 1 of what ld64 read.
__device__ __forceinline__ F2 pair(const uint32_t (&v)[2][32], int e) {
    return f2(__uint_as_float(v[e >> 4][2 * (e & 15)]), __uint_as_float(v[e >> 4][2 * (e & 15) + 1]));
}

// Dot product of eight bf16 pairs; sum over groups of L lanes.
__device__ __forceinline__ float dot8(uint4 a, uint4 b) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        sum = fmaf(__uint_as_float(x[e] << 16), __uint_as_float(y[e] << 16), sum);
        sum = fmaf(__uint_as_float(x[e] & 0xFFFF0000u), __uint_as_float(y[e] & 0xFFFF0000u), sum);
    }
    return sum;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}

// x = P (x - delta) for a row's 64 columns; zeros after column `last`; to TMEM in bf16, over the first 32 columns.
__device__ __forceinline__ void gradient_of_scores(uint32_t (&x)[2][32], const F2 (&pr)[32], F2 minus_delta) {
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        const float2 q = parts(mul(pr[e], add2(pair(x, e), minus_delta)));
        x[e >> 4][2 * (e & 15)] = __float_as_uint(q.x);
        x[e >> 4][2 * (e & 15) + 1] = __float_as_uint(q.y);
    }
}
__device__ __forceinline__ void mask_after(uint32_t (&x)[2][32], int last) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (c * 32 + e > last) x[c][e] = 0u;
}
__device__ __forceinline__ void store_scores(uint32_t taddr, const uint32_t (&x)[2][32]) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t o[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
            o[e] = pack_bf16x2(__uint_as_float(x[c][2 * e]), __uint_as_float(x[c][2 * e + 1]));
        tmem_st16(taddr + c * 16, o);
    }
}

// Adds a row's 64 gradients of scores, in fp32 before their rounding.
__device__ __forceinline__ void add_row(F2 (&sum)[2], const uint32_t (&x)[2][32]) {
#pragma unroll
    for (int e = 0; e < 32; ++e) sum[e & 1] = add2(sum[e & 1], pair(x, e));
}
__device__ __forceinline__ float total(const F2 (&sum)[2]) {
    const float2 q = parts(add2(sum[0], sum[1]));
    return q.x + q.y;
}

// ---------------------------------------------------------------------------------------------------------------
// dQ
// ---------------------------------------------------------------------------------------------------------------

template <int DP>
struct CfgQ {
    static constexpr int kBoxes = DP / 64;
    static constexpr uint32_t kTileBytes = kBoxes * 16384u;
    // a K tile is held from its scores to its gradients, a V tile for one product
    static constexpr int kStagesK = 3, kStagesV = 2;
    static constexpr size_t kSmem = 1024 + (2 + kStagesK + kStagesV) * static_cast<size_t>(kTileBytes) + 512 + 256;
};

template <int DP, int N>
__global__ void __launch_bounds__(kThreads, 1)
attn_dq_kernel(const __grid_constant__ AttnBwdParams p, const __grid_constant__ AttnSeqs<N> seqs) {
    const int item = attn_item();
    if (item >= p.sh.items) return;   // the last plane of the grid
    using C = CfgQ<DP>;
    constexpr int SK = C::kStagesK, SV = C::kStagesV;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_1024(smem_raw);
    uint8_t* sQ = smem;
    uint8_t* sDO = sQ + C::kTileBytes;
    uint8_t* sK = sDO + C::kTileBytes;
    uint8_t* sV = sK + SK * C::kTileBytes;
    float* sDelta = reinterpret_cast<float*>(sV + SV * C::kTileBytes);   // 128
    uint64_t* bars = reinterpret_cast<uint64_t*>(sDelta + 128);
    uint64_t* q_full = bars;
    uint64_t* do_full = q_full + 1;
    uint64_t* o_full = do_full + 1;
    uint64_t* o_read = o_full + 1;
    uint64_t* k_full = o_read + 1;        // SK each
    uint64_t* k_empty = k_full + SK;
    uint64_t* v_full = k_empty + SK;       // SV each
    uint64_t* v_empty = v_full + SV;
    uint64_t* s_full = v_empty + SV;       // 2 score buffers
    uint64_t* dp_full = s_full + 2;
    uint64_t* ds_full = dp_full + 1;
    uint64_t* dq_full = ds_full + 1;
    uint64_t* k_fixed = dq_full + 1;
    uint64_t* dp_read = k_fixed + 1;
    uint64_t* drain = dp_read + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    __shared__ int abort_flag;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const AttnShape& sh = p.sh;
    const AttnSeq sq = find_seq(seqs, sh.n_seqs, item);
    const int tpt = kAttnTile >> sh.hp_log2;
    const int tiles = (sq.ql + tpt - 1) >> (7 - sh.hp_log2);
    const int local = item - sq.item0;
    const int tok0 = (tiles - 1 - local) * tpt;
    const int head0 = blockIdx.x << sh.hp_log2;
    const int kvh = sh.hp == sh.group ? blockIdx.x : head0 / sh.group;
    const int off = sq.kl - sq.ql;
    const int last = min(tok0 + tpt, sq.ql) - 1 + off;            // last key the tile sees
    const int n = last >= 0 ? last / kAttnTile + 1 : 0;
    const bool tail = n * kAttnTile > sq.kl;

    const auto load_k = [&](int j) {
        const int s = j % SK;
        mbar_arrive_expect_tx(&k_full[s], C::kTileBytes);
        for (int b = 0; b < C::kBoxes; ++b)
            tma_load_3d(sK + s * C::kTileBytes + b * 16384, &p.mapK, &k_full[s], b * 64, kvh, sq.k0 + j * kAttnTile);
    };
    const auto load_v = [&](int j) {
        const int s = j % SV;
        mbar_arrive_expect_tx(&v_full[s], C::kTileBytes);
        for (int b = 0; b < C::kBoxes; ++b)
            tma_load_3d(sV + s * C::kTileBytes + b * 16384, &p.mapV, &v_full[s], b * 64, kvh, sq.k0 + j * kAttnTile);
    };
    uint8_t* const sO = sK + (SK - 1) * C::kTileBytes;   // O, for delta, where a later K tile goes
    // the first loads are under way before the CTA is set up
    const int ahead = min(SV, n);
    if (warp == 8) {
        if (lane == 0) {
            tma_prefetch_desc(&p.mapQ);
            tma_prefetch_desc(&p.mapK);
            tma_prefetch_desc(&p.mapV);
            tma_prefetch_desc(&p.mapDO);
            mbar_init(q_full, 1);
            mbar_init(do_full, 1);
            mbar_init(o_full, 1);
            mbar_init(o_read, 256);
            tma_prefetch_desc(&p.mapO);
            for (int s = 0; s < SK; ++s) {
                mbar_init(&k_full[s], 1);
                mbar_init(&k_empty[s], 1);
            }
            for (int s = 0; s < SV; ++s) {
                mbar_init(&v_full[s], 1);
                mbar_init(&v_empty[s], 1);
            }
            mbar_init(&s_full[0], 1);
            mbar_init(&s_full[1], 1);
            mbar_init(dp_full, 1);
            mbar_init(ds_full, 256);
            mbar_init(dq_full, 1);
            mbar_init(k_fixed, 1);
            mbar_init(dp_read, 256);
            mbar_init(drain, 1);
            abort_flag = 0;
            fence_barrier_init();
            pdl_wait();
            if (n > 0) {
                mbar_arrive_expect_tx(q_full, C::kTileBytes);
                for (int b = 0; b < C::kBoxes; ++b)
                    tma_load_3d(sQ + b * 16384, &p.mapQ, q_full, b * 64, head0, sq.q0 + tok0);
                load_k(0);
                mbar_arrive_expect_tx(do_full, C::kTileBytes);
                for (int b = 0; b < C::kBoxes; ++b)
                    tma_load_3d(sDO + b * 16384, &p.mapDO, do_full, b * 64, head0, sq.q0 + tok0);
                load_v(0);
                mbar_arrive_expect_tx(o_full, C::kTileBytes);
                for (int b = 0; b < C::kBoxes; ++b)
                    tma_load_3d(sO + b * 16384, &p.mapO, o_full, b * 64, head0, sq.q0 + tok0);
            }
            for (int j = 1; j < ahead; ++j) {
                load_k(j);
                load_v(j);
            }
        }
        __syncwarp();
    } else if (warp == 9) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_trigger();
    const uint32_t tmem = *tmem_slot;
    const uint32_t t_s = tmem, t_dp = tmem + 256, t_dq = tmem + 384;
    const WaitCtx w{&abort_flag, p.ctl.status, p.ctl.wait_ns, kKAttnDq << 8};

    if (warp == 8) {
        bool ok = true;
        int issued = ahead;
        for (int j = ahead; j < n; ++j) {
            if (lane == 0) {
                ok = mbar_wait(&k_empty[j % SK], ((j / SK) & 1) ^ 1u, w, 1);
                if (ok && j == SK - 1) ok = mbar_wait(o_read, 0, w, 15);
                if (ok) {
                    load_k(j);
                    ok = mbar_wait(&v_empty[j % SV], ((j / SV) & 1) ^ 1u, w, 2);
                    if (ok)
                        load_v(j);
                    else
                        mbar_wait_drain(&k_full[j % SK], (j / SK) & 1, p.ctl.wait_ns);
                }
            }
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (!ok) break;
            ++issued;
        }
        if (ok && tail && n > 0) {
            const int s = (n - 1) % SK;
            ok = mbar_wait(&k_full[s], ((n - 1) / SK) & 1, w, 3);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (ok) {
                zero_tile_rows(sK + s * C::kTileBytes, C::kBoxes, sq.kl - (n - 1) * kAttnTile);
                __syncwarp();
                if (lane == 0) mbar_arrive(k_fixed);
            }
        }
        if (lane == 0) {
            // every copy lands before the CTA exits, also when another warp gave up
            if (n > 0) {
                mbar_wait_drain(q_full, 0, p.ctl.wait_ns);
                mbar_wait_drain(do_full, 0, p.ctl.wait_ns);
                mbar_wait_drain(o_full, 0, p.ctl.wait_ns);
            }
            for (int j = max(0, issued - SK); j < issued; ++j) mbar_wait_drain(&k_full[j % SK], (j / SK) & 1, p.ctl.wait_ns);
            for (int j = max(0, issued - SV); j < issued; ++j) mbar_wait_drain(&v_full[j % SV], (j / SV) & 1, p.ctl.wait_ns);
        }
    } else if (warp == 9) {
        if (elect_one()) {
            const uint32_t idesc_s = make_idesc_bf16(128, 128, false, false);
            const uint32_t idesc_q = make_idesc_bf16(128, sh.d16, false, true);
            const uint64_t qd = make_smem_desc(smem_u32(sQ), 16, 1024, kSw128);
            const uint64_t dod = make_smem_desc(smem_u32(sDO), 16, 1024, kSw128);
            const uint64_t kd = make_smem_desc(smem_u32(sK), 16, 1024, kSw128);
            const uint64_t kmn = make_smem_desc(smem_u32(sK), 16384, 1024, kSw128);
            const uint64_t vd = make_smem_desc(smem_u32(sV), 16, 1024, kSw128);
            bool ok = true;
            if (n > 0) ok = mbar_wait(q_full, 0, w, 4);
            // turn j: S(j) (its own buffer), dP(j) as soon as the score warps hold dP(j - 1) in registers, then
            // dQ += dS(j - 1) K(j - 1): dP(j) is formed while they work on dS(j - 1)
            for (int j = 0; j <= n && n > 0 && ok; ++j) {
                if (j < n) {
                    if (!mbar_wait(&k_full[j % SK], (j / SK) & 1, w, 5)) { ok = false; break; }
                    if (tail && j == n - 1 && !mbar_wait(k_fixed, 0, w, 6)) { ok = false; break; }
                    tc_fence_after();
                    mma_rows<DP>(t_s + (j & 1) * 128, qd, kd + static_cast<uint64_t>(j % SK) * (C::kTileBytes >> 4), idesc_s);
                    umma_commit(&s_full[j & 1]);
                    if (j == 0 && !mbar_wait(do_full, 0, w, 13)) { ok = false; break; }
                    if (!mbar_wait(&v_full[j % SV], (j / SV) & 1, w, 7)) { ok = false; break; }
                    if (j > 0 && !mbar_wait(dp_read, (j - 1) & 1, w, 12)) { ok = false; break; }
                    tc_fence_after();
                    mma_rows<DP>(t_dp, dod, vd + static_cast<uint64_t>(j % SV) * (C::kTileBytes >> 4), idesc_s);
                    umma_commit(dp_full);
                    umma_commit(&v_empty[j % SV]);
                }
                if (j > 0) {
                    if (!mbar_wait(ds_full, (j - 1) & 1, w, 8)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t b = kmn + static_cast<uint64_t>((j - 1) % SK) * (C::kTileBytes >> 4);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        umma_bf16_ta(t_dq, t_s + ((j - 1) & 1) * 128 + a_col(ks), b + ks * 128u, idesc_q,
                                     (j != 1 || ks != 0) ? 1u : 0u);
                    umma_commit(&k_empty[(j - 1) % SK]);
                }
            }
            if (ok) umma_commit(dq_full);
            umma_commit(drain);
            mbar_wait_drain(drain, 0, p.ctl.wait_ns);
        }
        __syncwarp();
    } else {
        const int g = warp >> 2;                     // columns [64 g, 64 g + 64) of every tile
        const int quad = warp & 3;
        const int r = quad * 32 + lane;
        const int tok = tok0 + (r >> sh.hp_log2);
        const int head = head0 + (r & (sh.hp - 1));
        const bool row_ok = tok < sq.ql;
        const int limit = tok + off;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const float sl = sh.scale_log2;
        // under the first loads
        if (sq.gap + sh.lead + sh.trail > 0)
            fill_rows<16>(p.dQ, nullptr, nullptr, sh, head0, sh.hp_log2, static_cast<int64_t>(sq.q0) + sq.ql, sq.gap,
                      local, tiles, item, sh.items, threadIdx.x);
        const int64_t at = (static_cast<int64_t>(sq.q0) + tok) * sh.hq + head;
        // a row that is not there, or sees no key: every score is masked below
        const float lse2 = row_ok && limit >= 0 ? p.lse[at] * kLog2e : 0.f;
        bool ok = true;
        const F2 sl2 = f2(sl, sl), lse22 = f2(-lse2, -lse2);
        F2 delta2 = f2(0.f, 0.f), rest[2] = {delta2, delta2};
        for (int j = 0; j < n; ++j) {
            const uint32_t ts = t_s + (j & 1) * 128 + lanes + g * 64;
            ok = mbar_wait(&s_full[j & 1], (j >> 1) & 1, w, 9);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok && j > 0) break;   // the first turn has a barrier of all score warps
            tc_fence_after();
            uint32_t x[2][32];
            F2 pr[32];
            ld64(ts, x);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const float2 q = parts(fma2(pair(x, e), sl2, lse22));
                pr[e] = f2(ex2(q.x), ex2(q.y));
            }
            if (j == 0) {
                // delta of the tile's rows: needed from here on
                ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(do_full, 0, w, 14) && mbar_wait(o_full, 0, w, 16));
                // DP / 8 lanes a row, 8 features a lane
                constexpr int kLanes = DP / 8, kRows = 256 / kLanes, kSteps = 128 / kRows;
                const int sub = threadIdx.x % kLanes, first = threadIdx.x / kLanes;
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const int dr = k * kRows + first;
                    const uint32_t at_ = (sub >> 3) * 16384 + dr * 128 + (((sub & 7) ^ (dr & 7)) << 4);
                    const uint4 a = lds128(smem_u32(sO) + at_), b = lds128(smem_u32(sDO) + at_);
                    const float sum = lanes_sum<kLanes>(dot8(a, b));
                    if (sub == 0) sDelta[dr] = sum;
                }
                mbar_arrive(o_read);
                score_sync<256>();
                if (!ok) break;
                const float delta = sDelta[r];
                delta2 = f2(-delta, -delta);
            }
            ok = mbar_wait(dp_full, j & 1, w, 10);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after();
            ld64(t_dp + lanes + g * 64, x);
            tc_fence_before();
            mbar_arrive(dp_read);
            gradient_of_scores(x, pr, delta2);
            if ((j + 1) * kAttnTile - 1 > tok0 + off) mask_after(x, limit - j * kAttnTile - g * 64);
            store_scores(ts, x);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(ds_full);
            add_row(rest, x);
        }
        if (ok && n > 0) {
            ok = mbar_wait(dq_full, 0, w, 11);
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc_fence_after();
        }
        if (n > 0) {
            // delta for the next pass (every thread has read its own: all arrived for the last product); all score warps
            // come here, also after a wait that ran out
            if (g == 1) sDelta[r] = total(rest);
            score_sync<256>();
            if (row_ok && g == 0) p.delta[at] = total(rest) + sDelta[r] - parts(delta2).x;
        }
        if (ok) {
            // group g features [64 g, 64 g + 64), through Q's shared memory: all products are done
            store_tile(p.dQ.p + (static_cast<int64_t>(sq.q0) + tok0) * p.dQ.row + static_cast<int64_t>(head0) * p.dQ.head +
                               g * 64, p.dQ.row, p.dQ.head, sh.hp_log2, (sq.ql - tok0) << sh.hp_log2, sh.d - g * 64,
                           min(max(sh.d16 - g * 64, 0), 64), smem_u32(sQ) + g * 16384, t_dq + lanes + g * 64, quad, n > 0, sh.scale);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------------------------------------------
// dQ over few keys
// ---------------------------------------------------------------------------------------------------------------

// The same pass with key tiles of 64, four score warps and half the shared memory and TMEM: two CTAs an SM, one of which
// works while the other starts (its first tiles take 5000 cycles) or ends.  A product of 64 columns with both operands
// in shared memory costs 3/4 of one of 128, so long ranges are slower.  us (before the sums for delta, 1% here) for 8192 tokens with 32/8 heads of 128 in
// samples of 77, 128, 256, 450, 1024, 2048, 4096 tokens: 86, 78, 83, 100, 135, 204, 343 against 119, 100, 100, 115, 136,
// 186, 276 with tiles of 128; 32 heads of 64 the same way (58 against 83 at 128, 256 against 233 at 4096).
constexpr int kShortKeys = 64;
constexpr int kShortThreads = 192;   // warps 0-3: scores and gradients of scores; warp 4: TMA; warp 5: MMAs

template <int DP>
struct CfgShort {
    static constexpr int kBoxes = DP / 64;
    static constexpr uint32_t kTileBytes = kBoxes * 16384u, kKeyBytes = kTileBytes / 2;
    static constexpr int kStagesK = 2;
    static constexpr size_t kSmem = 2 * static_cast<size_t>(kTileBytes) + (kStagesK + 1) * static_cast<size_t>(kKeyBytes) + 512 + 256;
};

template <int DP, int N>
__global__ void __launch_bounds__(kShortThreads, 2)
attn_dq_short_kernel(const __grid_constant__ AttnBwdParams p, const __grid_constant__ AttnSeqs<N> seqs) {
    const int item = attn_item();
    if (item >= p.sh.items) return;   // the last plane of the grid
    using C = CfgShort<DP>;
    constexpr int SK = C::kStagesK, KT = kShortKeys;
    // no other shared memory: the dynamic part starts on a swizzle atom, and there is no room to move it
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw;
    if ((smem_u32(smem) & 1023u) != 0) {
        if (threadIdx.x == 0 && p.ctl.status) atomicCAS(p.ctl.status, 0, (kKAttnDq << 8) | 0xFF);
        return;
    }
    uint8_t* sQ = smem;
    uint8_t* sDO = sQ + C::kTileBytes;
    uint8_t* sK = sDO + C::kTileBytes;
    uint8_t* sV = sK + SK * C::kKeyBytes;
    float* sDelta = reinterpret_cast<float*>(sV + C::kKeyBytes);   // 128
    uint64_t* bars = reinterpret_cast<uint64_t*>(sDelta + 128);
    uint64_t* q_full = bars;
    uint64_t* do_full = q_full + 1;
    uint64_t* k_full = do_full + 1;        // SK each
    uint64_t* k_empty = k_full + SK;
    uint64_t* v_full = k_empty + SK;
    uint64_t* v_empty = v_full + 1;
    uint64_t* s_full = v_empty + 1;
    uint64_t* dp_full = s_full + 1;
    uint64_t* ds_full = dp_full + 1;
    uint64_t* dq_full = ds_full + 1;
    uint64_t* k_fixed = dq_full + 1;
    uint64_t* dp_read = k_fixed + 1;
    uint64_t* drain = dp_read + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    int& abort_flag = *reinterpret_cast<int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const AttnShape& sh = p.sh;
    const AttnSeq sq = find_seq(seqs, sh.n_seqs, item);
    const int tpt = kAttnTile >> sh.hp_log2;
    const int tiles = (sq.ql + tpt - 1) >> (7 - sh.hp_log2);
    const int local = item - sq.item0;
    const int tok0 = (tiles - 1 - local) * tpt;
    const int head0 = blockIdx.x << sh.hp_log2;
    const int kvh = sh.hp == sh.group ? blockIdx.x : head0 / sh.group;
    const int off = sq.kl - sq.ql;
    const int last = min(tok0 + tpt, sq.ql) - 1 + off;            // last key the tile sees
    const int n = last >= 0 ? last / KT + 1 : 0;
    const bool tail = n * KT > sq.kl;

    const auto load_k = [&](int j) {
        const int s = j % SK;
        mbar_arrive_expect_tx(&k_full[s], C::kKeyBytes);
        for (int b = 0; b < C::kBoxes; ++b)
            tma_load_3d(sK + s * C::kKeyBytes + b * 8192, &p.mapK, &k_full[s], b * 64, kvh, sq.k0 + j * KT);
    };
    const auto load_v = [&](int j) {
        mbar_arrive_expect_tx(v_full, C::kKeyBytes);
        for (int b = 0; b < C::kBoxes; ++b)
            tma_load_3d(sV + b * 8192, &p.mapV, v_full, b * 64, kvh, sq.k0 + j * KT);
    };
    // O, of which delta needs the rows: DP / 8 lanes a row, 8 features a lane
    constexpr int kLanes = DP / 8, kRows = 128 / kLanes, kSteps = 128 / kRows;
    const int dsub = threadIdx.x % kLanes, dfirst = threadIdx.x / kLanes;
    uint4 o_rows[kSteps];
    if (warp == 4) {
        if (lane == 0) {
            tma_prefetch_desc(&p.mapQ);
            tma_prefetch_desc(&p.mapK);
            tma_prefetch_desc(&p.mapV);
            tma_prefetch_desc(&p.mapDO);
            mbar_init(q_full, 1);
            mbar_init(do_full, 1);
            for (int s = 0; s < SK; ++s) {
                mbar_init(&k_full[s], 1);
                mbar_init(&k_empty[s], 1);
            }
            mbar_init(v_full, 1);
            mbar_init(v_empty, 1);
            mbar_init(s_full, 1);
            mbar_init(dp_full, 1);
            mbar_init(ds_full, 128);
            mbar_init(dq_full, 1);
            mbar_init(k_fixed, 1);
            mbar_init(dp_read, 128);
            mbar_init(drain, 1);
            abort_flag = 0;
            fence_barrier_init();
            pdl_wait();
            if (n > 0) {
                mbar_arrive_expect_tx(q_full, C::kTileBytes);
                for (int b = 0; b < C::kBoxes; ++b)
                    tma_load_3d(sQ + b * 16384, &p.mapQ, q_full, b * 64, head0, sq.q0 + tok0);
                load_k(0);
                mbar_arrive_expect_tx(do_full, C::kTileBytes);
                for (int b = 0; b < C::kBoxes; ++b)
                    tma_load_3d(sDO + b * 16384, &p.mapDO, do_full, b * 64, head0, sq.q0 + tok0);
                load_v(0);
            }
        }
        __syncwarp();
    } else if (warp == 5) {
        tmem_alloc(tmem_slot, 256);
        tmem_relinquish();
    } else if (n > 0) {
        pdl_wait();
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int dr = k * kRows + dfirst, dt = tok0 + (dr >> sh.hp_log2), dh = head0 + (dr & (sh.hp - 1));
            o_rows[k] = make_uint4(0u, 0u, 0u, 0u);
            if (dt < sq.ql && dsub * 8 < sh.d)
                o_rows[k] = *reinterpret_cast<const uint4*>(p.O.p + (static_cast<int64_t>(sq.q0) + dt) * p.O.row +
                                                            dh * p.O.head + dsub * 8);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_trigger();
    const uint32_t tmem = *tmem_slot;
    // two buffers of 64 columns: turn j has S(j) (then dS(j)) in buffer j & 1 and dP(j) in the other
    const uint32_t t_dq = tmem + 128;
    const WaitCtx w{&abort_flag, p.ctl.status, p.ctl.wait_ns, kKAttnDq << 8};

    if (warp == 4) {
        bool ok = true;
        const int ahead = min(1, n);
        int issued = ahead, issued_v = ahead;
        for (int j = ahead; j < n; ++j) {
            if (lane == 0) {
                ok = mbar_wait(&k_empty[j % SK], ((j / SK) & 1) ^ 1u, w, 1);
                if (ok) {
                    load_k(j);
                    ++issued;
                    ok = mbar_wait(v_empty, (j & 1) ^ 1u, w, 2);
                    if (ok) {
                        load_v(j);
                        ++issued_v;
                    }
                }
            }
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (!ok) break;
        }
        if (ok && tail && n > 0) {
            const int s = (n - 1) % SK;
            ok = mbar_wait(&k_full[s], ((n - 1) / SK) & 1, w, 3);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (ok) {
                zero_tile_rows<KT>(sK + s * C::kKeyBytes, C::kBoxes, sq.kl - (n - 1) * KT);
                __syncwarp();
                if (lane == 0) mbar_arrive(k_fixed);
            }
        }
        if (lane == 0) {
            // every copy lands before the CTA exits, also when another warp gave up
            if (n > 0) {
                mbar_wait_drain(q_full, 0, p.ctl.wait_ns);
                mbar_wait_drain(do_full, 0, p.ctl.wait_ns);
            }
            for (int j = max(0, issued - SK); j < issued; ++j) mbar_wait_drain(&k_full[j % SK], (j / SK) & 1, p.ctl.wait_ns);
            if (issued_v > 0) mbar_wait_drain(v_full, (issued_v - 1) & 1, p.ctl.wait_ns);
        }
    } else if (warp == 5) {
        if (elect_one()) {
            const uint32_t idesc_s = make_idesc_bf16(128, KT, false, false);
            const uint32_t idesc_q = make_idesc_bf16(128, sh.d16, false, true);
            const uint64_t qd = make_smem_desc(smem_u32(sQ), 16, 1024, kSw128);
            const uint64_t dod = make_smem_desc(smem_u32(sDO), 16, 1024, kSw128);
            const uint64_t kd = make_smem_desc(smem_u32(sK), 16, 1024, kSw128);
            const uint64_t kmn = make_smem_desc(smem_u32(sK), 8192, 1024, kSw128);
            const uint64_t vd = make_smem_desc(smem_u32(sV), 16, 1024, kSw128);
            const auto k_ready = [&](int j) {
                return mbar_wait(&k_full[j % SK], (j / SK) & 1, w, 5) && (!tail || j != n - 1 || mbar_wait(k_fixed, 0, w, 6));
            };
            const auto at = [&](int j) { return tmem + (j & 1) * 64; };
            bool ok = n > 0 && mbar_wait(q_full, 0, w, 4) && k_ready(0);
            if (ok) {
                tc_fence_after();
                mma_rows<DP, KT>(at(0), qd, kd, idesc_s);
                umma_commit(s_full);
                ok = mbar_wait(do_full, 0, w, 13) && mbar_wait(v_full, 0, w, 7);
            }
            if (ok) {
                tc_fence_after();
                mma_rows<DP, KT>(at(1), dod, vd, idesc_s);
                umma_commit(dp_full);
                umma_commit(v_empty);
            }
            // turn j: S(j + 1) as soon as dP(j) has been read from its buffer, dQ += dS(j) K(j), then dP(j + 1) over dS(j)
            for (int j = 0; j < n && ok; ++j) {
                if (j + 1 < n) {
                    if (!k_ready(j + 1) || !mbar_wait(dp_read, j & 1, w, 12)) { ok = false; break; }
                    tc_fence_after();
                    mma_rows<DP, KT>(at(j + 1), qd, kd + static_cast<uint64_t>((j + 1) % SK) * (C::kKeyBytes >> 4), idesc_s);
                    umma_commit(s_full);
                }
                if (!mbar_wait(ds_full, j & 1, w, 8)) { ok = false; break; }
                tc_fence_after();
                const uint64_t b = kmn + static_cast<uint64_t>(j % SK) * (C::kKeyBytes >> 4);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    umma_bf16_ta(t_dq, at(j) + ks * 8, b + ks * 128u, idesc_q, (j != 0 || ks != 0) ? 1u : 0u);
                umma_commit(&k_empty[j % SK]);
                if (j + 1 < n) {
                    if (!mbar_wait(v_full, (j + 1) & 1, w, 7)) { ok = false; break; }
                    tc_fence_after();
                    mma_rows<DP, KT>(at(j), dod, vd, idesc_s);
                    umma_commit(dp_full);
                    umma_commit(v_empty);
                }
            }
            if (ok) umma_commit(dq_full);
            umma_commit(drain);
            mbar_wait_drain(drain, 0, p.ctl.wait_ns);
        }
        __syncwarp();
    } else {
        const int r = warp * 32 + lane;
        const int tok = tok0 + (r >> sh.hp_log2);
        const int head = head0 + (r & (sh.hp - 1));
        const bool row_ok = tok < sq.ql;
        const int limit = tok + off;
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
        const float sl = sh.scale_log2;
        const int64_t at = (static_cast<int64_t>(sq.q0) + tok) * sh.hq + head;
        // a row that is not there, or sees no key: every score is masked below
        const float lse2 = row_ok && limit >= 0 ? p.lse[at] * kLog2e : 0.f;
        // under the first loads
        if (sq.gap + sh.lead + sh.trail > 0)
            fill_rows<8>(p.dQ, nullptr, nullptr, sh, head0, sh.hp_log2, static_cast<int64_t>(sq.q0) + sq.ql, sq.gap,
                         local, tiles, item, sh.items, threadIdx.x);
        bool ok = true;
        float delta = 0.f;
        if (n > 0) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(do_full, 0, w, 14));
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const int dr = k * kRows + dfirst;
                const uint4 b = lds128(smem_u32(sDO) + (dsub >> 3) * 16384 + dr * 128 + (((dsub & 7) ^ (dr & 7)) << 4));
                const float sum = lanes_sum<kLanes>(dot8(o_rows[k], b));
                if (dsub == 0) sDelta[dr] = sum;
            }
            score_sync<128>();
            delta = sDelta[r];
        }
        F2 rest[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
        const F2 sl2 = f2(sl, sl), lse22 = f2(-lse2, -lse2), delta2 = f2(-delta, -delta);
        for (int j = 0; ok && j < n; ++j) {
            const uint32_t ts = tmem + (j & 1) * 64 + lanes, tdp = tmem + ((j + 1) & 1) * 64 + lanes;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(s_full, j & 1, w, 9));
            if (!ok) break;
            tc_fence_after();
            uint32_t x[2][32];
            F2 pr[32];
            ld64(ts, x);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const float2 q = parts(fma2(pair(x, e), sl2, lse22));
                pr[e] = f2(ex2(q.x), ex2(q.y));
            }
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(dp_full, j & 1, w, 10));
            if (!ok) break;
            tc_fence_after();
            ld64(tdp, x);
            tc_fence_before();
            mbar_arrive(dp_read);
            gradient_of_scores(x, pr, delta2);
            if ((j + 1) * KT - 1 > tok0 + off) mask_after(x, limit - j * KT);
            store_scores(ts, x);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(ds_full);
            add_row(rest, x);
        }
        if (row_ok && n > 0) p.delta[at] = delta + total(rest);   // for the next pass
        if (ok && n > 0) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(dq_full, 0, w, 11));
            tc_fence_after();
        }
        if (ok)
            // through Q's shared memory: all products are done
            store_tile(p.dQ.p + (static_cast<int64_t>(sq.q0) + tok0) * p.dQ.row + static_cast<int64_t>(head0) * p.dQ.head,
                       p.dQ.row, p.dQ.head, sh.hp_log2, (sq.ql - tok0) << sh.hp_log2, sh.d, sh.d16, smem_u32(sQ),
                       t_dq + lanes, warp, n > 0, sh.scale);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

// ---------------------------------------------------------------------------------------------------------------
// dK, dV
// ---------------------------------------------------------------------------------------------------------------

template <int DP>
struct CfgKV {
    static constexpr int kBoxes = DP / 64;
    static constexpr uint32_t kTileBytes = kBoxes * 16384u;
    // a Q tile is held from its scores to dK, a dO tile from dP to dV
    static constexpr int kStagesQ = 3, kStagesO = 2;
    static constexpr size_t kSmem = (2 + kStagesQ + kStagesO) * static_cast<size_t>(kTileBytes) + 2 * 2 * 512 + 256;
};

template <int DP, int N>
__global__ void __launch_bounds__(kThreads, 1)
attn_dkdv_kernel(const __grid_constant__ AttnBwdParams p, const __grid_constant__ AttnSeqs<N> seqs) {
    const int item = attn_item();
    if (item >= p.sh.items) return;   // the last plane of the grid
    using C = CfgKV<DP>;
    constexpr int SQ = C::kStagesQ, SO = C::kStagesO;
    // no other shared memory: the dynamic part starts on a swizzle atom, and there is no room to move it
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw;
    if ((smem_u32(smem) & 1023u) != 0) {
        if (threadIdx.x == 0 && p.ctl.status) atomicCAS(p.ctl.status, 0, (kKAttnDkDv << 8) | 0xFF);
        return;
    }
    uint8_t* sK = smem;
    uint8_t* sV = sK + C::kTileBytes;
    uint8_t* sQ = sV + C::kTileBytes;
    uint8_t* sDO = sQ + SQ * C::kTileBytes;
    float* sStat = reinterpret_cast<float*>(sDO + SO * C::kTileBytes);   // [2][-lse2 128, -delta 128]
    uint64_t* bars = reinterpret_cast<uint64_t*>(sStat + 2 * 256);
    uint64_t* k_full = bars;               // K
    uint64_t* v_full = k_full + 1;         // V
    uint64_t* q_full = v_full + 1;         // SQ each
    uint64_t* q_empty = q_full + SQ;
    uint64_t* q_fixed = q_empty + SQ;      // Q rows past the sequence are zero
    uint64_t* do_full = q_fixed + SQ;      // SO each
    uint64_t* do_empty = do_full + SO;
    uint64_t* do_fixed = do_empty + SO;
    uint64_t* s_full = do_fixed + SO;
    uint64_t* dp_full = s_full + 1;
    uint64_t* p_full = dp_full + 1;
    uint64_t* ds_full = p_full + 1;
    uint64_t* out_full = ds_full + 1;
    uint64_t* stat_full = out_full + 1;    // the next tile's statistics are in shared memory
    uint64_t* drain = stat_full + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    int& abort_flag = *reinterpret_cast<int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const AttnShape& sh = p.sh;
    const AttnSeq sq = find_seq(seqs, sh.n_seqs, item);
    const int tpt = kAttnTile >> sh.hp_log2;
    // the first key tiles have the most queries; of a sequence with split queries the item has piece `piece` of a tile's
    int kt = item - sq.item0, piece = 0;
    if (sq.split)
        for (int c = (sq.kl + kAttnTile - 1) / kAttnTile; kt >= c; c = attn_tiles_over(sq, sh, piece * p.most)) {
            kt -= c;
            ++piece;
        }
    const int kvh = blockIdx.x;
    const int off = sq.kl - sq.ql;
    const int key0 = kt * kAttnTile;
    // the first query tile with a row that sees the first key, and the tiles after it, for each pack of the group
    const int i0 = max(0, key0 - off) >> (7 - sh.hp_log2);
    const int qt = (sq.ql + tpt - 1) >> (7 - sh.hp_log2);
    const int per = max(0, qt - i0);
    const int packs = sh.group >> sh.hp_log2;
    const int all = per * packs;
    const int pieces = sq.split ? max(1, (all + p.most - 1) / p.most) : 1, each = (all + pieces - 1) / pieces;
    const int t0 = piece * each, n = min(each, all - t0);   // the item's turns
    const int ragged = sq.ql - (qt - 1) * tpt;           // tokens of the last query tile
    const bool tail = ragged < tpt;

    const auto head_of = [&](int t) { return kvh * sh.group + ((packs == 1 ? 0 : (t0 + t) / per) << sh.hp_log2); };
    const auto tile_of = [&](int t) { return i0 + (packs == 1 ? t0 + t : (t0 + t) % per); };
    const auto load_q = [&](int t) {
        const int s = t % SQ;
        mbar_arrive_expect_tx(&q_full[s], C::kTileBytes);
        for (int b = 0; b < C::kBoxes; ++b)
            tma_load_3d(sQ + s * C::kTileBytes + b * 16384, &p.mapQ, &q_full[s], b * 64, head_of(t), sq.q0 + tile_of(t) * tpt);
    };
    const auto load_do = [&](int t) {
        const int s = t % SO;
        mbar_arrive_expect_tx(&do_full[s], C::kTileBytes);
        for (int b = 0; b < C::kBoxes; ++b)
            tma_load_3d(sDO + s * C::kTileBytes + b * 16384, &p.mapDO, &do_full[s], b * 64, head_of(t), sq.q0 + tile_of(t) * tpt);
    };
    // the first loads are under way before the CTA's other warps are set up
    const int ahead = min(SO, n);
    if (warp == 8) {
        if (lane == 0) {
            tma_prefetch_desc(&p.mapQ);
            tma_prefetch_desc(&p.mapK);
            tma_prefetch_desc(&p.mapV);
            tma_prefetch_desc(&p.mapDO);
            mbar_init(k_full, 1);
            mbar_init(v_full, 1);
            for (int s = 0; s < SQ; ++s) {
                mbar_init(&q_full[s], 1);
                mbar_init(&q_empty[s], 1);
                mbar_init(&q_fixed[s], 1);
            }
            for (int s = 0; s < SO; ++s) {
                mbar_init(&do_full[s], 1);
                mbar_init(&do_empty[s], 1);
                mbar_init(&do_fixed[s], 1);
            }
            mbar_init(s_full, 1);
            mbar_init(dp_full, 1);
            mbar_init(p_full, 256);
            mbar_init(ds_full, 256);
            mbar_init(out_full, 1);
            mbar_init(stat_full, 256);
            mbar_init(drain, 1);
            abort_flag = 0;
            fence_barrier_init();
            pdl_wait();
            if (n > 0) {
                mbar_arrive_expect_tx(k_full, C::kTileBytes);
                for (int b = 0; b < C::kBoxes; ++b)
                    tma_load_3d(sK + b * 16384, &p.mapK, k_full, b * 64, kvh, sq.k0 + key0);
                load_q(0);
                mbar_arrive_expect_tx(v_full, C::kTileBytes);
                for (int b = 0; b < C::kBoxes; ++b)
                    tma_load_3d(sV + b * 16384, &p.mapV, v_full, b * 64, kvh, sq.k0 + key0);
                load_do(0);
            }
            for (int t = 1; t < ahead; ++t) {
                load_q(t);
                load_do(t);
            }
        }
        __syncwarp();
    } else if (warp == 9) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_trigger();
    const uint32_t tmem = *tmem_slot;
    const uint32_t t_s = tmem, t_dp = tmem + 128, t_dv = tmem + 256, t_dk = tmem + 256 + DP;
    const WaitCtx w{&abort_flag, p.ctl.status, p.ctl.wait_ns, kKAttnDkDv << 8};

    if (warp == 8) {
        bool ok = true;
        int issued = ahead, issued_o = ahead;
        const auto fix = [&](uint8_t* tile, uint64_t* full, uint32_t ph, uint64_t* fixed, bool ragged_tile, int site) {
            if (ragged_tile) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(full, ph, w, site));
                if (!ok) return;
                zero_tile_rows(tile, C::kBoxes, ragged << sh.hp_log2);
                __syncwarp();
            }
            // the MMAs of every tile wait here: its rows are the sequence's own
            if (lane == 0) mbar_arrive(fixed);
        };
        for (int t = 0; t < n; ++t) {
            const int s = t % SQ, o = t % SO;
            const bool ragged_tile = tail && tile_of(t) == qt - 1;
            if (t >= ahead) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(&q_empty[s], ((t / SQ) & 1) ^ 1u, w, 1));
                if (!ok) break;
                if (lane == 0) load_q(t);
                ++issued;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(&do_empty[o], ((t / SO) & 1) ^ 1u, w, 2));
                if (!ok) break;
                if (lane == 0) load_do(t);
                ++issued_o;
            }
            fix(sQ + s * C::kTileBytes, &q_full[s], (t / SQ) & 1, &q_fixed[s], ragged_tile, 3);
            if (!ok) break;
            fix(sDO + o * C::kTileBytes, &do_full[o], (t / SO) & 1, &do_fixed[o], ragged_tile, 4);
            if (!ok) break;
        }
        if (lane == 0) {
            // every copy lands before the CTA exits, also when another warp gave up
            if (n > 0) {
                mbar_wait_drain(k_full, 0, p.ctl.wait_ns);
                mbar_wait_drain(v_full, 0, p.ctl.wait_ns);
            }
            for (int t = max(0, issued - SQ); t < issued; ++t) mbar_wait_drain(&q_full[t % SQ], (t / SQ) & 1, p.ctl.wait_ns);
            for (int t = max(0, issued_o - SO); t < issued_o; ++t) mbar_wait_drain(&do_full[t % SO], (t / SO) & 1, p.ctl.wait_ns);
        }
    } else if (warp == 9) {
        if (elect_one()) {
            const uint32_t idesc_s = make_idesc_bf16(128, 128, false, false);
            const uint32_t idesc_o = make_idesc_bf16(128, sh.d16, false, true);
            const uint64_t kd = make_smem_desc(smem_u32(sK), 16, 1024, kSw128);
            const uint64_t vd = make_smem_desc(smem_u32(sV), 16, 1024, kSw128);
            const uint64_t qd = make_smem_desc(smem_u32(sQ), 16, 1024, kSw128);
            const uint64_t dod = make_smem_desc(smem_u32(sDO), 16, 1024, kSw128);
            const uint64_t qmn = make_smem_desc(smem_u32(sQ), 16384, 1024, kSw128);
            const uint64_t domn = make_smem_desc(smem_u32(sDO), 16384, 1024, kSw128);
            bool ok = true;
            if (n > 0) ok = mbar_wait(k_full, 0, w, 5);
            // turn t: dV += P(t - 1)^T dO(t - 1), S^T(t), dK += dS(t - 1)^T Q(t - 1), dP^T(t)
            for (int t = 0; t <= n && n > 0 && ok; ++t) {
                if (t > 0) {
                    if (!mbar_wait(p_full, (t - 1) & 1, w, 10)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t b = domn + static_cast<uint64_t>((t - 1) % SO) * (C::kTileBytes >> 4);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        umma_bf16_ta(t_dv, t_s + a_col(ks), b + ks * 128u, idesc_o, (t != 1 || ks != 0) ? 1u : 0u);
                    umma_commit(&do_empty[(t - 1) % SO]);
                }
                if (t < n) {
                    if (!mbar_wait(&q_full[t % SQ], (t / SQ) & 1, w, 6)) { ok = false; break; }
                    if (!mbar_wait(&q_fixed[t % SQ], (t / SQ) & 1, w, 7)) { ok = false; break; }
                    tc_fence_after();
                    mma_rows<DP>(t_s, kd, qd + static_cast<uint64_t>(t % SQ) * (C::kTileBytes >> 4), idesc_s);
                    umma_commit(s_full);
                }
                if (t > 0) {
                    if (!mbar_wait(ds_full, (t - 1) & 1, w, 11)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t b = qmn + static_cast<uint64_t>((t - 1) % SQ) * (C::kTileBytes >> 4);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        umma_bf16_ta(t_dk, t_dp + a_col(ks), b + ks * 128u, idesc_o, (t != 1 || ks != 0) ? 1u : 0u);
                    umma_commit(&q_empty[(t - 1) % SQ]);
                }
                if (t < n) {
                    if (t == 0 && !mbar_wait(v_full, 0, w, 8)) { ok = false; break; }
                    if (!mbar_wait(&do_full[t % SO], (t / SO) & 1, w, 9)) { ok = false; break; }
                    if (!mbar_wait(&do_fixed[t % SO], (t / SO) & 1, w, 8)) { ok = false; break; }
                    tc_fence_after();
                    mma_rows<DP>(t_dp, vd, dod + static_cast<uint64_t>(t % SO) * (C::kTileBytes >> 4), idesc_s);
                    umma_commit(dp_full);
                }
            }
            if (ok) umma_commit(out_full);
            umma_commit(drain);
            mbar_wait_drain(drain, 0, p.ctl.wait_ns);
        }
        __syncwarp();
    } else {
        const int g = warp >> 2;
        const int quad = warp & 3;
        const int r = quad * 32 + lane;              // key of the tile
        const int ct = threadIdx.x & 127;            // the query row whose statistics this thread fetches
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t ts = t_s + lanes + g * 64;
        const uint32_t tdp = t_dp + lanes + g * 64;
        const float sl = sh.scale_log2;
        const float* src = g == 0 ? p.lse : p.delta; // group 0 fetches lse, group 1 delta
        const F2 sl2 = f2(sl, sl);
        // two tiles ahead: lse (a row that is not there, or sees no key: +inf, P = 0) or delta
        const auto fetch = [&](int t) -> float {
            const int tok = tile_of(t) * tpt + (ct >> sh.hp_log2);
            const int head = head_of(t) + (ct & (sh.hp - 1));
            const bool there = t < n && tok < sq.ql && tok + off >= 0;
            float x = g == 0 ? -neg_inf() : 0.f;
            if (there) x = src[(static_cast<int64_t>(sq.q0) + tok) * sh.hq + head];
            return x;
        };
        const float unit = g == 0 ? -kLog2e : -1.f;   // applied when it is stored: the load is not waited for before
        if (sq.gap + sh.lead + sh.trail > 0)
            fill_rows<16>(p.dK, &p.dV, nullptr, sh, kvh, 0, static_cast<int64_t>(sq.k0) + sq.kl, piece == 0 ? sq.gap : 0, kt,
                      (sq.kl + kAttnTile - 1) / kAttnTile, item, sh.items, threadIdx.x);
        bool ok = true;
        // statistics of tile t in buffer t & 1: tile 0's now, each later one's in the turn before
        sStat[g * 128 + ct] = n > 0 ? fetch(0) * unit : 0.f;
        mbar_arrive(stat_full);
        float next = n > 0 ? fetch(1) : 0.f;
        for (int t = 0; t < n; ++t) {
            float* stat = sStat + (t & 1) * 256;
            const int i = tile_of(t);
            const uint32_t st = smem_u32(stat) + g * 256;    // this group's 64 columns
            ok = mbar_wait(s_full, t & 1, w, 12);
            ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(stat_full, t & 1, w, 15));
            if (!ok) break;
            tc_fence_after();
            uint32_t v[2][32], x[2][32];
            ld64(ts, v);
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const uint4 q = lds128(st + (c * 32 + e) * 4);
                    const float2 a = parts(fma2(f2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])), sl2,
                                                f2(__uint_as_float(q.x), __uint_as_float(q.y))));
                    const float2 b = parts(fma2(f2(__uint_as_float(v[c][e + 2]), __uint_as_float(v[c][e + 3])), sl2,
                                                f2(__uint_as_float(q.z), __uint_as_float(q.w))));
                    v[c][e] = __float_as_uint(ex2(a.x));
                    v[c][e + 1] = __float_as_uint(ex2(a.y));
                    v[c][e + 2] = __float_as_uint(ex2(b.x));
                    v[c][e + 3] = __float_as_uint(ex2(b.y));
                }
            // keys after a query's limit: key0 + r > tok + off
            int cmin = 0;
            if (key0 + kAttnTile - 1 > i * tpt + off) {
                const int lo = key0 + r - off - i * tpt;     // first token of the tile that sees this key
                cmin = (max(lo, 0) << sh.hp_log2) - g * 64;
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c * 32 + e < cmin) v[c][e] = 0u;
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t o[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    o[e] = pack_bf16x2(__uint_as_float(v[c][2 * e]), __uint_as_float(v[c][2 * e + 1]));
                tmem_st16(ts + c * 16, o);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(p_full);
            // the other buffer is free once every warp is through with the tile before
            ok = t == 0 || mbar_wait(ds_full, (t - 1) & 1, w, 16);
            sStat[((t + 1) & 1) * 256 + g * 128 + ct] = next * unit;
            mbar_arrive(stat_full);
            next = fetch(t + 2);
            ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(dp_full, t & 1, w, 13));
            if (!ok) break;
            tc_fence_after();
            ld64(tdp, x);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t o[16];
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const uint4 q = lds128(st + 512 + (c * 32 + e) * 4);
                    const float2 a = parts(mul(f2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])),
                                               add2(f2(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])),
                                                    f2(__uint_as_float(q.x), __uint_as_float(q.y)))));
                    const float2 b = parts(mul(f2(__uint_as_float(v[c][e + 2]), __uint_as_float(v[c][e + 3])),
                                               add2(f2(__uint_as_float(x[c][e + 2]), __uint_as_float(x[c][e + 3])),
                                                    f2(__uint_as_float(q.z), __uint_as_float(q.w)))));
                    o[e / 2] = pack_bf16x2(a.x, a.y);
                    o[e / 2 + 1] = pack_bf16x2(b.x, b.y);
                }
                tmem_st16(tdp + c * 16, o);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(ds_full);
        }
        if (ok && n > 0) {
            ok = mbar_wait(out_full, 0, w, 14);
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc_fence_after();
        }
        if (ok && pieces > 1) {
            float* const slot = p.part + (static_cast<int64_t>(sq.split - 1 + item - sq.item0) * sh.hkv + kvh) * kAttnKvSlotFloats + g * 128 * 128;
#pragma unroll 1
            for (int c = 0; c < sh.d16; c += 16) {
                uint32_t o[16];
                tmem_ld16((g == 0 ? t_dv : t_dk) + lanes + c, o);
                tmem_ld_wait(o);
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    stg128(slot + ((c + e) * 128 + r * 4), make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]));
            }
        } else if (ok) {
            // group 0 writes dV, group 1 dK, through V's and K's shared memory: all products are done
            const AttnMat& m = g == 0 ? p.dV : p.dK;
            store_tile(m.p + (static_cast<int64_t>(sq.k0) + key0) * m.row + static_cast<int64_t>(kvh) * m.head, m.row, m.head,
                           0, sq.kl - key0, sh.d, sh.d16, smem_u32(g == 0 ? sV : sK), (g == 0 ? t_dv : t_dk) + lanes, quad, n > 0,
                           g == 0 ? 1.f : sh.scale);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the partial dK and dV of the key tiles whose queries were split, in the pieces' order.  A block a key tile, a key/value
// head and eight features of dV or dK, a thread a row.
template <int N>
__global__ void __launch_bounds__(128) attn_kv_join_kernel(const __grid_constant__ AttnBwdParams p, const __grid_constant__ AttnSeqs<N> seqs) {
    pdl_wait();
    pdl_trigger();
    const AttnShape& sh = p.sh;
    int i = 0, kt = blockIdx.y;
    for (int c; kt >= (c = (seqs.s[i].kl + kAttnTile - 1) / kAttnTile); ++i) kt -= c;
    const AttnSeq& sq = seqs.s[i];
    const int pieces = (attn_turns(sq, sh, kt) + p.most - 1) / p.most;
    const int r = threadIdx.x, key = kt * kAttnTile + r;
    if (pieces < 2 || key >= sq.kl) return;
    const int groups = sh.d / 8, which = blockIdx.z / groups, c = (blockIdx.z - which * groups) * 8;   // dV, dK
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    int at = sq.split - 1 + kt;
    for (int q = 0; q < pieces; ++q) {
        const float* const x = p.part + (static_cast<int64_t>(at) * sh.hkv + blockIdx.x) * kAttnKvSlotFloats + which * 128 * 128 + c * 128 + r * 4;
        const float4 a = *reinterpret_cast<const float4*>(x), b = *reinterpret_cast<const float4*>(x + 4 * 128);
        o[0] += a.x, o[1] += a.y, o[2] += a.z, o[3] += a.w;
        o[4] += b.x, o[5] += b.y, o[6] += b.z, o[7] += b.w;
        at += q == 0 ? (sq.kl + kAttnTile - 1) / kAttnTile : attn_tiles_over(sq, sh, q * p.most);
    }
    const AttnMat& m = which == 0 ? p.dV : p.dK;
    const float f = which == 0 ? 1.f : sh.scale;
    stg128(m.p + (static_cast<int64_t>(sq.k0) + key) * m.row + static_cast<int64_t>(blockIdx.x) * m.head + c,
           make_uint4(pack_bf16x2(o[0] * f, o[1] * f), pack_bf16x2(o[2] * f, o[3] * f), pack_bf16x2(o[4] * f, o[5] * f),
                      pack_bf16x2(o[6] * f, o[7] * f)));
}

template <int DP, int N>
cudaError_t run_dq_short(const AttnBwdParams& p, const AttnSeqs<kAttnMaxSeqs>& seqs, cudaStream_t stream) {
    return launch_pdl(attn_dq_short_kernel<DP, N>, attn_grid(p.sh.packs, p.sh.items), dim3(kShortThreads), CfgShort<DP>::kSmem,
                      stream, p, reinterpret_cast<const AttnSeqs<N>&>(seqs));
}

template <int DP, int N>
cudaError_t run_dq(const AttnBwdParams& p, const AttnSeqs<kAttnMaxSeqs>& seqs, cudaStream_t stream) {
    return launch_pdl(attn_dq_kernel<DP, N>, attn_grid(p.sh.packs, p.sh.items), dim3(kThreads), CfgQ<DP>::kSmem, stream, p,
                      reinterpret_cast<const AttnSeqs<N>&>(seqs));
}

template <int DP, int N>
cudaError_t run_dkdv(const AttnBwdParams& p, const AttnSeqs<kAttnMaxSeqs>& seqs, cudaStream_t stream) {
    return launch_pdl(attn_dkdv_kernel<DP, N>, attn_grid(p.sh.hkv, p.sh.items), dim3(kThreads), CfgKV<DP>::kSmem, stream, p,
                      reinterpret_cast<const AttnSeqs<N>&>(seqs));
}

template <int DP, int N>
cudaError_t configure() {
    cudaError_t e = cudaFuncSetAttribute(attn_dq_kernel<DP, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(CfgQ<DP>::kSmem));
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(attn_dq_short_kernel<DP, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(CfgShort<DP>::kSmem));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(attn_dkdv_kernel<DP, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(CfgKV<DP>::kSmem));
}

}  // namespace

cudaError_t attn_bwd_configure() {
    cudaError_t e = configure<64, kAttnFewSeqs>();
    if (e == cudaSuccess) e = configure<64, kAttnMaxSeqs>();
    if (e == cudaSuccess) e = configure<128, kAttnFewSeqs>();
    if (e == cudaSuccess) e = configure<128, kAttnMaxSeqs>();
    return e;
}

cudaError_t launch_attn_dq(const AttnBwdParams& p, const AttnSeqs<kAttnMaxSeqs>& seqs, bool short_keys, cudaStream_t stream) {
    const bool few = p.sh.n_seqs <= kAttnFewSeqs;
    if (short_keys) {
        if (p.sh.d <= 64) return few ? run_dq_short<64, kAttnFewSeqs>(p, seqs, stream) : run_dq_short<64, kAttnMaxSeqs>(p, seqs, stream);
        return few ? run_dq_short<128, kAttnFewSeqs>(p, seqs, stream) : run_dq_short<128, kAttnMaxSeqs>(p, seqs, stream);
    }
    if (p.sh.d <= 64) return few ? run_dq<64, kAttnFewSeqs>(p, seqs, stream) : run_dq<64, kAttnMaxSeqs>(p, seqs, stream);
    return few ? run_dq<128, kAttnFewSeqs>(p, seqs, stream) : run_dq<128, kAttnMaxSeqs>(p, seqs, stream);
}

cudaError_t launch_attn_dkdv(const AttnBwdParams& p, const AttnSeqs<kAttnMaxSeqs>& seqs, cudaStream_t stream) {
    const bool few = p.sh.n_seqs <= kAttnFewSeqs;
    if (p.sh.d <= 64)
        return few ? run_dkdv<64, kAttnFewSeqs>(p, seqs, stream) : run_dkdv<64, kAttnMaxSeqs>(p, seqs, stream);
    return few ? run_dkdv<128, kAttnFewSeqs>(p, seqs, stream) : run_dkdv<128, kAttnMaxSeqs>(p, seqs, stream);
}

cudaError_t launch_attn_kv_join(const AttnBwdParams& p, const AttnSeqs<kAttnMaxSeqs>& seqs, int n, int tiles, cudaStream_t stream) {
    const dim3 grid(p.sh.hkv, tiles, 2 * (p.sh.d / 8));
    if (n <= kAttnFewSeqs)
        return launch_pdl(attn_kv_join_kernel<kAttnFewSeqs>, grid, dim3(128), 0, stream, p,
                          reinterpret_cast<const AttnSeqs<kAttnFewSeqs>&>(seqs));
    return launch_pdl(attn_kv_join_kernel<kAttnMaxSeqs>, grid, dim3(128), 0, stream, p, seqs);
}

}  // namespace lora
