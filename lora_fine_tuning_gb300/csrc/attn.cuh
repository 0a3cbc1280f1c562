// Device-side pieces shared by the packed-attention kernels.
#pragma once

#include "attn.h"
#include "common.cuh"
#include "f32x2.cuh"

namespace lora {

// D[tmem] (+)= A[tmem] * B[smem]: A's rows are lanes, each 32-bit column holds two consecutive K elements (bf16).
__device__ __forceinline__ void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// True in one lane of a converged warp, the same one every time.  MMAs issued under it take a few cycles each; under
// `lane == 0`, where the assembler cannot see that one thread of a uniform branch runs, each took about 90 (traced in the
// forward kernel) and its operands went wrong where a run-time branch stood between two of them.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "elect.sync _|p, 0xFFFFFFFF;\n"
        "selp.b32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(p));
    return p != 0;
}

// One product of 128 x kBRows values over DP features, both operands K-major tiles of 64-feature boxes.  Every K step is
// issued, past the head's width too (the tiles hold zeros there): no branch stands between the steps.
template <int DP, int kBRows = 128>
__device__ __forceinline__ void mma_rows(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc) {
#pragma unroll
    for (int ks = 0; ks < DP / 16; ++ks) {
        const uint64_t h = static_cast<uint64_t>(ks >> 2), kk = static_cast<uint64_t>(ks & 3);
        umma_bf16(d_tmem, a + h * 1024u + kk * 2u, b + h * (kBRows * 8u) + kk * 2u, idesc, ks != 0 ? 1u : 0u);
    }
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Thread i of the warp writes row (lane base + i), 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Waits for this thread's TMEM loads.  The loaded registers pass through an asm statement after the wait: arithmetic on
// them, which the compiler may otherwise place before the wait, then depends on it (a load still in flight would land
// in a register that already serves another purpose).
template <int N>
__device__ __forceinline__ void tmem_landed(uint32_t (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                          "+r"(r[i + 6]), "+r"(r[i + 7])::"memory");
}
template <int N>
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[N]) {
    tmem_ld_wait();
    tmem_landed(r);
}
template <int M, int N>
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[M][N]) {
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < M; ++i) tmem_landed(r[i]);
}

// A CTA's work item (tile); gridDim.x counts the heads, and gridDim.y alone may not count a long batch's tiles.
__device__ __forceinline__ int attn_item() { return blockIdx.z * gridDim.y + blockIdx.y; }

// The sequence that holds work item `item`: the last whose first item is not after it.  By a converged warp, a lane an
// entry: first every 32nd entry of a long table, then the 32 from there.
template <int N>
__device__ __forceinline__ AttnSeq find_seq(const AttnSeqs<N>& t, int n, int item) {
    const int lane = lane_id();
    int from = 0;
    if (N > 32 && n > 32) {
        const int at = lane * 32;
        from = (__popc(__ballot_sync(0xFFFFFFFFu, at < n && t.s[min(at, n - 1)].item0 <= item)) - 1) * 32;
    }
    const int at = from + lane;
    const int k = from + __popc(__ballot_sync(0xFFFFFFFFu, at < n && t.s[min(at, n - 1)].item0 <= item)) - 1;
    return t.s[max(k, 0)];
}

// Zeroes rows [from, R) of a swizzled tile of `boxes` 64-feature boxes of R rows x 128 bytes, by one warp (rows
// past the end of a sequence belong to another sequence or to nobody: a probability of zero times what lies there
// would still be a NaN when it is infinite or NaN).  The caller orders it before the MMAs that read the tile.
template <int R = 128>
__device__ __forceinline__ void zero_tile_rows(uint8_t* tile, int boxes, int from) {
    const uint32_t base = smem_u32(tile);
    const int n = (R - from) * 8;
    for (int b = 0; b < boxes; ++b)
        for (int i = lane_id(); i < n; i += 32)
            sts128(base + b * (R * 128) + from * 128 + i * 16, make_uint4(0u, 0u, 0u, 0u));
    fence_proxy_async_smem();
}

// Rows of an output tile that a warp holds in TMEM (row quad * 32 + lane at `taddr`, `have` false: zeros) times f, in bf16,
// to global memory: tile row r is token r >> hp_log2 of `out`, head r & (hp - 1); rows from `rows` on are not written.
// They pass through shared memory (`stage`: boxes of 128 rows x 64 features, 16-byte chunks swizzled by the row), so that
// eight lanes store 128 bytes of a row together.  A row a lane made every store touch 32 lines: 5100 cycles a tile.
__device__ __forceinline__ void store_tile(uint16_t* out, int64_t row_stride, int64_t head_stride, int hp_log2, int rows,
                                           int d, int d16, uint32_t stage, uint32_t taddr, int quad, bool have, float f) {
    const int lane = lane_id();
    const F2 ff = f2(f, f);
    if (rows <= quad * 32) return;
#pragma unroll 1
    for (int c = 0; c < d16; c += 64) {
        const uint32_t box = stage + (c >> 6) * 16384 + quad * 4096;
#pragma unroll
        for (int x = 0; x < 64; x += 32) {
            uint32_t o[32];
            if (have) {
                tmem_ld32(taddr + c + x, o);
                tmem_ld_wait(o);
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0u;
            }
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
                uint32_t q[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 v = parts(mul(f2(__uint_as_float(o[e + 2 * k]), __uint_as_float(o[e + 2 * k + 1])), ff));
                    q[k] = pack_bf16x2(v.x, v.y);
                }
                sts128(box + lane * 128 + ((((x + e) >> 3) ^ (lane & 7)) << 4), make_uint4(q[0], q[1], q[2], q[3]));
            }
        }
        __syncwarp();
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int row = k * 4 + (lane >> 3);
            v[k] = lds128(box + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
        }
        if (c + (lane & 7) * 8 < d) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int tr = quad * 32 + k * 4 + (lane >> 3);
                if (tr < rows)
                    stg128(out + static_cast<int64_t>(tr >> hp_log2) * row_stride +
                               static_cast<int64_t>(tr & ((1 << hp_log2) - 1)) * head_stride + c + (lane & 7) * 8, v[k]);
            }
        }
        __syncwarp();
    }
}

// Unused rows that an item fills: every tiles-th row of the gap after its sequence (from `after`), its share (item
// `turn` of `turns`) of the rows before the first and after the last sequence; heads [head0, head0 + hp) of a and, if
// there, b, and lse.  By 16 G threads, 16 a row and head.
template <int G>
static __device__ __noinline__ void fill_rows(const AttnMat& a, const AttnMat* b, float* lse, const AttnShape& sh, int head0,
                                              int hp_log2, int64_t after, int gap, int tile, int tiles, int turn, int turns,
                                              int thread) {
    const int hp = 1 << hp_log2, x = (thread & 15) * 8;
    const int h = (thread >> 4) & (hp - 1);
    constexpr int kLog = G == 16 ? 4 : 3;
    const int per = G >> min(hp_log2, kLog), mine = (thread >> 4) >> min(hp_log2, kLog);   // rows at a time
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const auto clear = [&](int64_t row) {
        for (int g = head0 + h; g < head0 + hp; g += G) {
            if (x < sh.d) {
                stg128(a.p + row * a.row + g * a.head + x, zero);
                if (b) stg128(b->p + row * b->row + g * b->head + x, zero);
            }
            if (lse && x == 0) lse[row * sh.hq + g] = neg_inf();
        }
    };
    for (int r = tile * per + mine; r < gap; r += tiles * per) clear(after + r);
    for (int r = turn * per + mine; r < sh.lead + sh.trail; r += turns * per)
        clear(r < sh.lead ? r : sh.trail0 + r - sh.lead);
}

}  // namespace lora
