// Forward of causal softmax attention over packed sequences with grouped heads.
//
//   S = scale Q K^T,  visible keys j <= i + (k_len - q_len),  lse_i = log sum_j exp S_ij,  O = exp(S - lse) V
//
// in one pass over the keys with the running maximum and sum of each row.  A CTA works on one 128-row query tile (tokens x
// heads of one group, attn.h); two CTAs share an SM: while the softmax of one runs, the tensor cores work on the other's
// products, and its start and end (about 10000 cycles) are covered, too.  Warps 0-3: the softmax, a thread one row; warp 4:
// TMA (K and V tiles of 128 keys through a ring of stages); warp 5: the MMAs.  S (fp32) lives in TMEM, is read by its
// row's thread, and P goes back in bf16 (the tensor cores' operand type; the sum is of the values before this rounding)
// over S's columns, from where the second product reads it as its A operand.
// The rows of O are rescaled in TMEM only when a row's maximum grew by more than 2^8 since the last rescaling (the
// statistics keep the older maximum until then: P stays below 2^8, far inside bf16's and fp32's ranges).
//
// Bound by the tensor cores and the chain S, softmax, P of two tiles: a turn of both takes 2870 cycles, their products
// 2048, each tile's softmax 1380.  8192 tokens with 32/8 heads of 128: 351 us (293 at the cuBLAS rate); four sequences of
// 4096 with 64/8 heads: 760 to 785 (587).  One CTA an SM with two query tiles that share K and V: 357 us, 77 us against
// 58 for samples of 77 tokens.
#include <algorithm>

#include "attn.cuh"
#include "kernels.h"

namespace lora {

namespace {

constexpr float kRescale = 8.f;   // log2 of the growth of a row's maximum that rescales O

constexpr int kThreads = 192;     // warps 0-3: softmax; warp 4: TMA; warp 5: MMAs

template <int DP>
struct Cfg {
    static constexpr int kBoxes = DP / 64;
    static constexpr uint32_t kTileBytes = kBoxes * 16384u;   // 128 rows x DP bf16
    static constexpr int kStages = DP == 128 ? 2 : 4;         // of K or V tiles, which alternate
    static constexpr size_t kSmem = 1024 + (1 + kStages) * static_cast<size_t>(kTileBytes) + 256;   // two CTAs an SM
};

template <int DP, int N>
__global__ void __launch_bounds__(kThreads, 2)
attn_fwd_kernel(const __grid_constant__ AttnFwdParams p, const __grid_constant__ AttnSeqs<N> seqs) {
    const int item = attn_item();
    if (item >= p.sh.items) return;   // the last plane of the grid
    using C = Cfg<DP>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_1024(smem_raw);
    uint8_t* sQ = smem;
    uint8_t* sKV = smem + C::kTileBytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + kStages * C::kTileBytes);
    uint64_t* q_full = bars;
    uint64_t* kv_full = q_full + 1;          // kStages
    uint64_t* kv_empty = kv_full + kStages;
    uint64_t* s_full = kv_empty + kStages;
    uint64_t* p_full = s_full + 1;           // 2: the halves of P
    uint64_t* o_full = p_full + 2;
    uint64_t* v_fixed = o_full + 1;          // the last V tile's rows past the sequence are zero
    uint64_t* drain = v_fixed + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    __shared__ int abort_flag;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    // the item: a query tile of one pack of heads, those with the most keys first
    const AttnShape& sh = p.sh;
    const AttnSeq sq = find_seq(seqs, sh.n_seqs, item);
    const int tpt = kAttnTile >> sh.hp_log2;                       // tokens in a tile
    const int tiles = attn_query_tiles(sq, sh);
    // of a sequence with split keys the item has piece `piece` of a tile's
    int local = item - sq.item0, piece = 0;
    if (sq.split)
        for (int c = tiles; local >= c; c = attn_tiles_seeing(sq, sh, piece * p.most)) {
            local -= c;
            ++piece;
        }
    const int tok0 = (tiles - 1 - local) * tpt;                     // first token
    const int head0 = blockIdx.x << sh.hp_log2;
    const int kvh = sh.hp == sh.group ? blockIdx.x : head0 / sh.group;
    const int off = sq.kl - sq.ql;
    const int all = attn_seen(sq, sh, tiles - 1 - local);           // its key tiles
    const int pieces = sq.split ? max(1, (all + p.most - 1) / p.most) : 1, each = (all + pieces - 1) / pieces;
    const int kb = piece * each, n = min(each, all - kb);           // the item's
    const bool tail = (kb + n) * kAttnTile > sq.kl;               // the last key tile ends past the sequence

    const auto load_kv = [&](int t) {
        const int s = t % kStages;
        mbar_arrive_expect_tx(&kv_full[s], C::kTileBytes);
        const CUtensorMap* map = (t & 1) ? &p.mapV : &p.mapK;
        for (int b = 0; b < C::kBoxes; ++b)
            tma_load_3d(sKV + s * C::kTileBytes + b * 16384, map, &kv_full[s], b * 64, kvh,
                        sq.k0 + (kb + (t >> 1)) * kAttnTile);
    };
    // the first loads are under way before the CTA's other warps are set up
    const int ahead = min(kStages, 2 * n);
    if (warp == 4) {
        if (lane == 0) {
            tma_prefetch_desc(&p.mapQ);
            tma_prefetch_desc(&p.mapK);
            tma_prefetch_desc(&p.mapV);
            mbar_init(q_full, 1);
            mbar_init(s_full, 1);
            mbar_init(&p_full[0], 128);
            mbar_init(&p_full[1], 128);
            mbar_init(o_full, 1);
            for (int s = 0; s < kStages; ++s) {
                mbar_init(&kv_full[s], 1);
                mbar_init(&kv_empty[s], 1);
            }
            mbar_init(v_fixed, 1);
            mbar_init(drain, 1);
            abort_flag = 0;
            fence_barrier_init();
            pdl_wait();
            if (n > 0) {
                mbar_arrive_expect_tx(q_full, C::kTileBytes);
                for (int b = 0; b < C::kBoxes; ++b)
                    tma_load_3d(sQ + b * 16384, &p.mapQ, q_full, b * 64, head0, sq.q0 + tok0);
            }
            for (int t = 0; t < ahead; ++t) load_kv(t);
        }
        __syncwarp();
    } else if (warp == 5) {
        tmem_alloc(tmem_slot, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_trigger();
    const uint32_t tmem = *tmem_slot;
    const WaitCtx w{&abort_flag, p.ctl.status, p.ctl.wait_ns, kKAttnFwd << 8};

    if (warp == 4) {
        bool ok = true;
        int issued = ahead;
        for (int t = ahead; t < 2 * n; ++t) {
            if (lane == 0) {
                ok = mbar_wait(&kv_empty[t % kStages], ((t / kStages) & 1) ^ 1u, w, 1);
                if (ok) load_kv(t);
            }
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (!ok) break;
            ++issued;
        }
        if (ok && tail && n > 0) {
            const int t = 2 * n - 1;
            ok = mbar_wait(&kv_full[t % kStages], (t / kStages) & 1, w, 2);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (ok) {
                zero_tile_rows(sKV + (t % kStages) * C::kTileBytes, C::kBoxes, sq.kl - (kb + n - 1) * kAttnTile);
                __syncwarp();
                if (lane == 0) mbar_arrive(v_fixed);
            }
        }
        if (lane == 0) {
            // every copy lands before the CTA exits, also when another warp gave up
            if (n > 0) mbar_wait_drain(q_full, 0, p.ctl.wait_ns);
            for (int t = max(0, issued - kStages); t < issued; ++t)
                mbar_wait_drain(&kv_full[t % kStages], (t / kStages) & 1, p.ctl.wait_ns);
        }
    } else if (warp == 5) {
        // the whole warp waits; one lane issues (elect_one)
        const uint32_t idesc_s = make_idesc_bf16(128, 128, false, false);
        const uint32_t idesc_o = make_idesc_bf16(128, sh.d16, false, true);
        const uint64_t qd = make_smem_desc(smem_u32(sQ), 16, 1024, kSw128);
        const uint64_t kd = make_smem_desc(smem_u32(sKV), 16, 1024, kSw128);       // K: rows x features
        const uint64_t vd = make_smem_desc(smem_u32(sKV), 16384, 1024, kSw128);    // V: features contiguous
        bool ok = true;
        const auto wait = [&](uint64_t* bar, uint32_t parity, int site) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, w, site));
            tc_fence_after();
            return ok;
        };
        // turn j: the product of P(j - 1) with V(j - 1), then the scores with K(j).  S(j) overwrites P(j - 1) in TMEM:
        // the MMAs execute in the order in which they are issued.
        for (int j = 0; j <= n && n > 0; ++j) {
            const int tk = 2 * j, tv = 2 * j - 1;
            if (j > 0) {
                const uint64_t b = vd + static_cast<uint64_t>(tv % kStages) * (C::kTileBytes >> 4);
                if (!wait(&kv_full[tv % kStages], (tv / kStages) & 1, 3)) break;
                if (tail && j == n && !wait(v_fixed, 0, 4)) break;
                if (j < n && !wait(&kv_full[tk % kStages], (tk / kStages) & 1, 5)) break;
                if (!wait(&p_full[0], (j - 1) & 1, 6)) break;
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        umma_bf16_ta(tmem + 128, tmem + ks * 8, b + ks * 128u, idesc_o, (j != 1 || ks != 0) ? 1u : 0u);
                }
                __syncwarp();
                if (!wait(&p_full[1], (j - 1) & 1, 8)) break;
                if (elect_one()) {
#pragma unroll
                    for (int ks = 4; ks < 8; ++ks)
                        umma_bf16_ta(tmem + 128, tmem + ks * 8, b + ks * 128u, idesc_o, 1u);
                    umma_commit(j == n ? o_full : &kv_empty[tv % kStages]);
                }
                __syncwarp();
            } else if (!wait(q_full, 0, 7) || !wait(&kv_full[0], 0, 5)) {
                break;
            }
            if (j < n) {
                if (elect_one()) {
                    mma_rows<DP>(tmem, qd, kd + static_cast<uint64_t>(tk % kStages) * (C::kTileBytes >> 4), idesc_s);
                    umma_commit(s_full);
                    umma_commit(&kv_empty[tk % kStages]);
                }
                __syncwarp();
            }
        }
        if (elect_one()) umma_commit(drain);
        __syncwarp();
        mbar_wait_drain(drain, 0, p.ctl.wait_ns);
        __syncwarp();
    } else {
        const int quad = warp;
        const int r = quad * 32 + lane;              // row of the tile = TMEM lane
        const int tok = tok0 + (r >> sh.hp_log2);
        const int head = head0 + (r & (sh.hp - 1));
        const int limit = tok + off;                 // last visible key (clamped below kl: tok < ql)
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        // under the first loads
        if (sq.gap + sh.lead + sh.trail > 0)
            fill_rows<8>(p.O, nullptr, p.lse, sh, head0, sh.hp_log2, static_cast<int64_t>(sq.q0) + sq.ql,
                      piece == 0 ? sq.gap : 0, local, tiles, item, sh.items, threadIdx.x);
        const uint32_t ts = tmem + lanes, to = ts + 128;
        const float sl = sh.scale_log2;
        const int first_limit = tok0 + off;          // last key the tile's first row sees
        float m = neg_inf(), l = 0.f;                // maximum (in the exponent's units) and sum
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            ok = mbar_wait(s_full, j & 1, w, 9);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after();
            uint32_t v[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, v[c]);
            tmem_ld_wait(v);
            if ((kb + j + 1) * kAttnTile - 1 > first_limit) {
                // keys past the row's limit (and past the sequence: limit < kl)
                const int lim = limit - (kb + j) * kAttnTile;
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c * 32 + e > lim) v[c][e] = 0xff800000u;
            }
            float tops[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                tops[c] = fmaxf(__uint_as_float(v[c][0]), __uint_as_float(v[c][1]));
#pragma unroll
                for (int e = 2; e < 32; e += 2)
                    tops[c] = max3(tops[c], __uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]));
            }
            const float top = sl * fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]);
            if (j == 0) {
                m = top;
            } else {
                const bool grow = top > m + kRescale;
                if (__any_sync(0xFFFFFFFFu, grow)) {
                    // s_full of this tile came after the previous product into O
                    const float mn = grow ? top : m;
                    const float f = grow ? (m == neg_inf() ? 0.f : ex2(m - mn)) : 1.f;
                    m = mn;
                    l *= f;
#pragma unroll 1
                    for (int c = 0; c < DP; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(to + c, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st16(to + c, o);
                    }
                    tmem_st_wait();
                }
            }
            const float ms = m == neg_inf() ? 0.f : m;   // a row without a visible key yet: exp2(-inf) = 0 throughout
            const F2 sl2 = f2(sl, sl), ms2 = f2(-ms, -ms);
            F2 sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
            // in halves of 64 keys: the product with V starts on the first while the second is computed
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int c = 2 * h; c < 2 * h + 2; ++c) {
                    uint32_t o[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 q = parts(fma2(f2(__uint_as_float(v[c][2 * e]), __uint_as_float(v[c][2 * e + 1])), sl2, ms2));
                        const float x = ex2(q.x), y = ex2(q.y);
                        sum[e & 1] = add2(sum[e & 1], f2(x, y));
                        o[e] = pack_bf16x2(x, y);
                    }
                    tmem_st16(ts + c * 16, o);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&p_full[h]);
            }
            const float2 q = parts(add2(sum[0], sum[1]));
            l += q.x + q.y;
        }
        if (ok && n > 0) {
            ok = mbar_wait(o_full, 0, w, 10);
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc_fence_after();
        }
        if (ok && pieces > 1) {
            float* const slot = p.part + (static_cast<int64_t>(sq.split - 1 + local * attn_pieces(sq, p.most) + piece) * sh.packs + blockIdx.x) * kAttnSlotFloats;
#pragma unroll 1
            for (int c = 0; c < sh.d16; c += 16) {
                uint32_t o[16];
                tmem_ld16(to + c, o);
                tmem_ld_wait(o);
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    stg128(slot + ((c + e) * 128 + r * 4), make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]));
            }
            slot[128 * 128 + r] = m;
            slot[128 * 128 + 128 + r] = l;
        } else if (ok) {
            // through the query tile's shared memory: its products are done
            const int rows = (sq.ql - tok0) << sh.hp_log2;    // of the tile that are in the sequence
            store_tile(p.O.p + (static_cast<int64_t>(sq.q0) + tok0) * p.O.row + static_cast<int64_t>(head0) * p.O.head,
                           p.O.row, p.O.head, sh.hp_log2, rows, sh.d, sh.d16, smem_u32(sQ), to, quad, n > 0,
                           l == 0.f ? 0.f : 1.f / l);   // no visible key: zeros; a NaN stays one
            if (r < rows)
                p.lse[(static_cast<int64_t>(sq.q0) + tok) * sh.hq + head] = l == 0.f ? neg_inf() : (m + __log2f(l)) * kLn2;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

// Joins the partial results of the tiles whose keys were split: with M the largest of their maxima m_s,
//   O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s.  Blocks of 128 rows x 4 features, a thread a row.
template <int N>
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ AttnFwdParams p,
                                                        const __grid_constant__ AttnSeqs<N> seqs) {
    pdl_wait();
    pdl_trigger();
    const AttnShape& sh = p.sh;
    int i = 0, u = blockIdx.y;   // tile, from the sequence's last
    for (int c; u >= (c = attn_query_tiles(seqs.s[i], sh)); ++i) u -= c;
    const AttnSeq& sq = seqs.s[i];
    const int tiles = attn_query_tiles(sq, sh), pieces = (attn_seen(sq, sh, tiles - 1 - u) + p.most - 1) / p.most;
    const int r = threadIdx.x, c = blockIdx.z * 4, tok = ((tiles - 1 - u) << (7 - sh.hp_log2)) + (r >> sh.hp_log2);
    if (pieces < 2 || tok >= sq.ql) return;
    const float* const slot = p.part + (static_cast<int64_t>(sq.split - 1 + u * attn_pieces(sq, p.most)) * sh.packs + blockIdx.x) * kAttnSlotFloats;
    const int64_t step = static_cast<int64_t>(sh.packs) * kAttnSlotFloats;
    float top = neg_inf();
    for (int s = 0; s < pieces; ++s) top = fmaxf(top, slot[s * step + 128 * 128 + r]);
    const float ts = top == neg_inf() ? 0.f : top;
    float l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < pieces; ++s) {
        const float* const q = slot + s * step;
        const float f = ex2(q[128 * 128 + r] - ts), ls = q[128 * 128 + 128 + r];
        if (ls == 0.f) continue;   // no key of this range is visible
        const float4 v = *reinterpret_cast<const float4*>(q + c * 128 + r * 4);
        l = fmaf(f, ls, l);
        o[0] = fmaf(f, v.x, o[0]);
        o[1] = fmaf(f, v.y, o[1]);
        o[2] = fmaf(f, v.z, o[2]);
        o[3] = fmaf(f, v.w, o[3]);
    }
    const float f = l == 0.f ? 0.f : 1.f / l;
    const int64_t row = static_cast<int64_t>(sq.q0) + tok;
    const int head = (blockIdx.x << sh.hp_log2) + (r & (sh.hp - 1));
    *reinterpret_cast<uint2*>(p.O.p + row * p.O.row + static_cast<int64_t>(head) * p.O.head + c) =
        make_uint2(pack_bf16x2(o[0] * f, o[1] * f), pack_bf16x2(o[2] * f, o[3] * f));
    if (c == 0) p.lse[row * sh.hq + head] = l == 0.f ? neg_inf() : (top + __log2f(l)) * kLn2;
}

// Rows of no sequence: zeros (and lse -inf), so that what reads the whole batch later finds no stale values.  A block takes
// as many rows at a time as its threads have 16-byte chunks for.
constexpr int kFillThreads = 256;
int fill_rows_at(int chunks) { return kFillThreads / std::min(chunks, kFillThreads); }

__global__ void __launch_bounds__(kFillThreads) attn_fill_kernel(const __grid_constant__ AttnFillParams p,
                                                                 const __grid_constant__ AttnGaps gaps) {
    pdl_wait();
    pdl_trigger();
    const int from = gaps.from[blockIdx.x], to = gaps.to[blockIdx.x];
    const int chunks = p.heads * (p.d / 8), lanes = min(chunks, kFillThreads), at = kFillThreads / lanes;
    const int sub = threadIdx.x / lanes, lane = threadIdx.x - sub * lanes;
    if (sub >= at) return;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    for (int row = from + blockIdx.y * at + sub; row < to; row += gridDim.y * at) {
        for (int c = lane; c < chunks; c += lanes) {
            const int h = c / (p.d / 8), x = (c - h * (p.d / 8)) * 8;
            stg128(p.a.p + static_cast<int64_t>(row) * p.a.row + static_cast<int64_t>(h) * p.a.head + x, z);
            if (p.b.p) stg128(p.b.p + static_cast<int64_t>(row) * p.b.row + static_cast<int64_t>(h) * p.b.head + x, z);
        }
        if (p.lse)
            for (int h = lane; h < p.heads; h += lanes) p.lse[static_cast<int64_t>(row) * p.heads + h] = neg_inf();
    }
}

template <int DP, int N>
cudaError_t run(const AttnFwdParams& p, const AttnSeqs<kAttnMaxSeqs>& seqs, cudaStream_t stream) {
    return launch_pdl(attn_fwd_kernel<DP, N>, attn_grid(p.sh.packs, p.sh.items), dim3(kThreads), Cfg<DP>::kSmem, stream, p,
                      reinterpret_cast<const AttnSeqs<N>&>(seqs));
}

template <int DP, int N>
cudaError_t configure() {
    return cudaFuncSetAttribute(attn_fwd_kernel<DP, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(Cfg<DP>::kSmem));
}

}  // namespace

cudaError_t attn_fwd_configure() {
    cudaError_t e = configure<64, kAttnFewSeqs>();
    if (e == cudaSuccess) e = configure<64, kAttnMaxSeqs>();
    if (e == cudaSuccess) e = configure<128, kAttnFewSeqs>();
    if (e == cudaSuccess) e = configure<128, kAttnMaxSeqs>();
    return e;
}

cudaError_t launch_attn_fwd(const AttnFwdParams& p, const AttnSeqs<kAttnMaxSeqs>& seqs, cudaStream_t stream) {
    const bool few = p.sh.n_seqs <= kAttnFewSeqs;
    if (p.sh.d <= 64) return few ? run<64, kAttnFewSeqs>(p, seqs, stream) : run<64, kAttnMaxSeqs>(p, seqs, stream);
    return few ? run<128, kAttnFewSeqs>(p, seqs, stream) : run<128, kAttnMaxSeqs>(p, seqs, stream);
}

cudaError_t launch_attn_join(const AttnFwdParams& p, const AttnSeqs<kAttnMaxSeqs>& seqs, int n, int tiles, cudaStream_t stream) {
    const dim3 grid(p.sh.packs, tiles, p.sh.d / 4);
    if (n <= kAttnFewSeqs)
        return launch_pdl(attn_join_kernel<kAttnFewSeqs>, grid, dim3(128), 0, stream, p,
                          reinterpret_cast<const AttnSeqs<kAttnFewSeqs>&>(seqs));
    return launch_pdl(attn_join_kernel<kAttnMaxSeqs>, grid, dim3(128), 0, stream, p, seqs);
}

cudaError_t launch_attn_fill(const AttnFillParams& p, const AttnGaps& gaps, cudaStream_t stream) {
    int longest = 1;
    for (int i = 0; i < p.n; ++i) longest = std::max(longest, gaps.to[i] - gaps.from[i]);
    // four rounds a block where that makes no more than 16 blocks an SM.  One gap of 8192 and of 262144 rows with 32 heads of
    // 128: 23 and 345 us with one token's attention; in 608 blocks 24 and 371, in 16 blocks 138 and 4030
    const int at = 4 * fill_rows_at(p.heads * (p.d / 8));
    const int blocks = std::max(1, std::min((longest + at - 1) / at, std::max(16, 16 * 152 / p.n)));
    return launch_pdl(attn_fill_kernel, dim3(p.n, blocks), dim3(kFillThreads), 0, stream, p, gaps);
}

}  // namespace lora
