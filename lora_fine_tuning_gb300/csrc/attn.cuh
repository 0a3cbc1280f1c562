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

// One 128 x 128 product over DP features, both operands K-major 128-row tiles of 64-feature boxes.  Every K step is
// issued, past the head's width too (the tiles hold zeros there): no branch stands between the steps.
template <int DP>
__device__ __forceinline__ void mma_rows(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc) {
#pragma unroll
    for (int ks = 0; ks < DP / 16; ++ks) {
        const uint64_t h = static_cast<uint64_t>(ks >> 2), kk = static_cast<uint64_t>(ks & 3);
        umma_bf16(d_tmem, a + h * 1024u + kk * 2u, b + h * 1024u + kk * 2u, idesc, ks != 0 ? 1u : 0u);
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

// The sequence that holds work item `item`: the last whose first item is not after it.
template <int N>
__device__ __forceinline__ AttnSeq find_seq(const AttnSeqs<N>& t, int n, int item) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.s[mid].item0 <= item) lo = mid;
        else hi = mid;
    }
    return t.s[lo];
}

// Zeroes rows [from, 128) of a swizzled tile of `boxes` 64-feature boxes of 128 rows x 128 bytes, by one warp (rows
// past the end of a sequence belong to another sequence or to nobody: a probability of zero times what lies there
// would still be a NaN when it is infinite or NaN).  The caller orders it before the MMAs that read the tile.
__device__ __forceinline__ void zero_tile_rows(uint8_t* tile, int boxes, int from) {
    const uint32_t base = smem_u32(tile);
    const int n = (128 - from) * 8;
    for (int b = 0; b < boxes; ++b)
        for (int i = lane_id(); i < n; i += 32)
            sts128(base + b * 16384 + from * 128 + i * 16, make_uint4(0u, 0u, 0u, 0u));
    fence_proxy_async_smem();
}

// 16 fp32 values -> 8 packed bf16 pairs, times f, to 16 consecutive output elements (8 at a time, features past d
// are not written; d % 8 == 0).
__device__ __forceinline__ void store_out16(uint16_t* out, const uint32_t (&v)[16], float f, int c0, int d) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(__uint_as_float(v[2 * i]) * f, __uint_as_float(v[2 * i + 1]) * f);
    if (c0 < d) stg128(out + c0, make_uint4(w[0], w[1], w[2], w[3]));
    if (c0 + 8 < d) stg128(out + c0 + 8, make_uint4(w[4], w[5], w[6], w[7]));
}

}  // namespace lora
