// Launch plans of the packed attention (k_attn_fwd.cu, k_attn_bwd.cu), filled by attn_api.cu.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "plan.h"

namespace lora {

constexpr int kAttnMaxSeqs = 1024;
constexpr int kAttnTile = 128;        // rows of a query tile and of a key tile

// One sequence of the batch.  A kernel's work items (tiles, attn_item()) are numbered sequence by sequence; item0 is the
// first of this one's (the table is in order of falling work, not of rows).  The heads are
// blockIdx.x: the tiles with the most work of all heads come first.
struct AttnSeq {
    int32_t q0, k0;      // first row of the queries, of the keys
    int32_t ql, kl;      // rows
    int32_t item0;
    int32_t gap;         // unused rows of the output after this sequence that its items fill
    int32_t split;       // keys (forward) or queries (dK and dV) split over several items: first slot + 1; 0: not split
};

// The table travels as a kernel parameter (no device table, no copy); a small batch passes a small one.
template <int N>
struct AttnSeqs {
    AttnSeq s[N];
};
constexpr int kAttnFewSeqs = 32;

// A matrix of rows x heads x d in global memory, strides in elements.
struct AttnMat {
    uint16_t* p;
    int64_t row, head;
};

// Query rows of one key/value head are tiled with the heads of its group: a 128-row tile holds 128 / hp tokens x hp
// query heads, row = token * hp + head, hp the largest power of two (at most 128) that divides the group.  The g / hp
// packs of a group are separate tiles.
struct AttnShape {
    int32_t n_seqs;
    int32_t items;           // tiles of all sequences
    int32_t hq, hkv, group;
    int32_t hp, hp_log2;     // query heads in a tile
    int32_t packs;           // hq / hp: packs of the whole layer
    int32_t d, d16;          // head width, rounded up to 16
    int32_t lead;            // unused rows [0, lead) and [trail0, trail0 + trail) of the output, filled by all items
    int32_t trail0, trail;
    float scale;             // softmax scale
    float scale_log2;        // scale * log2(e)
};

struct AttnFwdParams {
    CUtensorMap mapQ, mapK, mapV;
    AttnShape sh;
    AttnMat O;
    float* lse;              // rows x hq
    int32_t most;            // key tiles of an item of a sequence whose keys are split
    float* part;             // their partial results: slots of kAttnSlotFloats, slot * packs + pack
    DevCtl ctl;
};

// What an item of a split sequence leaves: the sums into O before their division, feature groups of 4 x 128 rows x 4,
// then each row's maximum and sum.
constexpr int kAttnSlotFloats = 128 * 128 + 2 * 128;
constexpr int kAttnMaxSlots = 640;   // slots x packs of a call: at most four items an SM (attn_api.cu)

struct AttnBwdParams {
    CUtensorMap mapQ, mapK, mapV, mapO, mapDO;
    AttnShape sh;
    const float* lse;        // rows x hq
    float* delta;            // rows x hq, from the first pass to the second
    int32_t most;            // query tiles of an item of a sequence whose queries are split for dK and dV
    float* part;             // their partial results: slots of kAttnKvSlotFloats, slot * hkv + head
    AttnMat O;
    AttnMat dQ, dK, dV;
    DevCtl ctl;
};

// Rows of the outputs that belong to no sequence: rows [from, to) of up to three matrices get zeros, lse -inf.
struct AttnGaps {
    int32_t from[kAttnMaxSeqs + 1], to[kAttnMaxSeqs + 1];
};
struct AttnFillParams {
    AttnMat a, b;            // b.p may be null
    int32_t heads, d;
    float* lse;              // may be null
    int32_t n;
};

// What an item of a sequence with split queries leaves: dV, then dK, each as feature groups of 4 x 128 rows x 4.
constexpr int kAttnKvSlotFloats = 2 * 128 * 128;

// Key tiles that query tile `tile` of a sequence sees, and the query tiles that see more than `n` of them; these are its last
// ones.  Items of a sequence with split keys: first one for every query tile, from the last, with up to `most` key tiles,
// then one for each that sees more than `most`, and so on.
__host__ __device__ inline int attn_query_tiles(const AttnSeq& q, const AttnShape& sh) {
    const int lg = 7 - sh.hp_log2;
    return (q.ql + (1 << lg) - 1) >> lg;
}
__host__ __device__ inline int attn_seen(const AttnSeq& q, const AttnShape& sh, int tile) {
    const int end = (tile + 1) << (7 - sh.hp_log2), last = (end < q.ql ? end : q.ql) - 1 + q.kl - q.ql;
    return last >= 0 ? last / kAttnTile + 1 : 0;
}
// Pieces of the keys of a sequence's last query tile: each of its tiles has as many slots.
__host__ __device__ inline int attn_pieces(const AttnSeq& q, int most) { return ((q.kl + kAttnTile - 1) / kAttnTile + most - 1) / most; }
__host__ __device__ inline int attn_tiles_seeing(const AttnSeq& q, const AttnShape& sh, int n) {
    if (q.ql == 0 || q.kl <= static_cast<int64_t>(n) * kAttnTile) return 0;
    const int lg = 7 - sh.hp_log2, tiles = attn_query_tiles(q, sh);
    // the first token that sees key n * 128, and its tile
    const int64_t token = static_cast<int64_t>(n) * kAttnTile - (q.kl - q.ql);
    return tiles - (token > 0 ? static_cast<int>(token >> lg) : 0);
}

// Key tiles of a sequence that more than `turns` query tiles (of all packs of a group) see; these are its first ones.
// Items of a sequence with split queries: first one for every key tile, with up to `most` query tiles, then one for each
// with more than `most`, and so on.
__host__ __device__ inline int attn_tiles_over(const AttnSeq& q, const AttnShape& sh, int turns) {
    const int lg = 7 - sh.hp_log2, qt = (q.ql + (1 << lg) - 1) >> lg;
    const int before = qt - turns / (sh.group >> sh.hp_log2);   // a key tile counts if its first query tile is before this
    const int64_t keys = before > 0 ? (static_cast<int64_t>(before) << lg) + q.kl - q.ql : 0;
    const int64_t seen = keys > 0 ? (keys + kAttnTile - 1) / kAttnTile : 0, all = (q.kl + kAttnTile - 1) / kAttnTile;
    return static_cast<int>(seen < all ? seen : all);
}
__host__ __device__ inline int attn_turns(const AttnSeq& q, const AttnShape& sh, int key_tile) {
    const int lg = 7 - sh.hp_log2, qt = (q.ql + (1 << lg) - 1) >> lg;
    const int first = key_tile * kAttnTile - (q.kl - q.ql);
    const int n = qt - ((first > 0 ? first : 0) >> lg);
    return (n > 0 ? n : 0) * (sh.group >> sh.hp_log2);
}

inline dim3 attn_grid(int heads, int items) {
    const int y = items < 65535 ? items : 65535;
    return dim3(static_cast<unsigned>(heads), static_cast<unsigned>(y), static_cast<unsigned>((items + y - 1) / y));
}

cudaError_t attn_fwd_configure();
cudaError_t attn_bwd_configure();
cudaError_t launch_attn_fwd(const AttnFwdParams& p, const AttnSeqs<kAttnMaxSeqs>& seqs, cudaStream_t stream);
// Joins the partial results of `tiles` query tiles, those of the first n sequences of the table.
cudaError_t launch_attn_join(const AttnFwdParams& p, const AttnSeqs<kAttnMaxSeqs>& seqs, int n, int tiles, cudaStream_t stream);
// short_keys: key tiles of 64, which mapK and mapV then describe.
cudaError_t launch_attn_dq(const AttnBwdParams& p, const AttnSeqs<kAttnMaxSeqs>& seqs, bool short_keys, cudaStream_t stream);
cudaError_t launch_attn_dkdv(const AttnBwdParams& p, const AttnSeqs<kAttnMaxSeqs>& seqs, cudaStream_t stream);
// Joins the partial results of `tiles` key tiles, those of the first n sequences of the table.
cudaError_t launch_attn_kv_join(const AttnBwdParams& p, const AttnSeqs<kAttnMaxSeqs>& seqs, int n, int tiles, cudaStream_t stream);
cudaError_t launch_attn_fill(const AttnFillParams& p, const AttnGaps& gaps, cudaStream_t stream);

}  // namespace lora
