// C ABI of the packed attention: validation, work items and launches.  See include/lora.h for the contract.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <utility>

#include "attn.h"
#include "host.h"

namespace lora {
namespace {

constexpr size_t kStatusBytes = 256;
constexpr size_t kSplitBytes = static_cast<size_t>(kAttnMaxSlots) * kAttnSlotFloats * 4;
constexpr int64_t kMaxKvSlots = kSplitBytes / 4 / kAttnKvSlotFloats;

struct Prepared {
    AttnShape sh;
    AttnSeqs<kAttnMaxSeqs> order;   // sequences with rows, most keys first
    int n = 0;
    AttnGaps q_gaps, k_gaps;
    int nq_gaps = 0, nk_gaps = 0;
};

lora_status check_mat(const void* p, const lora_attn_strides& s, int64_t rows, int heads, int d) {
    if (rows > 0 && !p) return LORA_EINVAL;
    if (!aligned16(p)) return LORA_EALIGN;
    if (s.row % 8 || s.head % 8) return LORA_EALIGN;
    if (s.row < 0 || s.head < 0 || s.row >= (int64_t{1} << 38) || s.head >= (int64_t{1} << 38)) return LORA_ESHAPE;
    // rows of heads, or heads of rows; either way no element twice
    const bool by_row = (heads == 1 || s.head >= d) && (rows <= 1 || s.row >= (heads - 1) * (heads == 1 ? 0 : s.head) + d);
    const bool by_head = (rows <= 1 || s.row >= d) && (heads == 1 || s.head >= (rows - 1) * s.row + d);
    return by_row || by_head ? LORA_OK : LORA_ESHAPE;
}

lora_status check_seqs(const lora_attn_seq* seqs, int32_t n, int64_t q_rows, int64_t k_rows, Prepared& c) {
    if (n < 0 || n > LORA_ATTN_MAX_SEQS) return LORA_ETABLE;
    if (n > 0 && !seqs) return LORA_EINVAL;
    int64_t q_end = 0, k_end = 0;
    c.n = c.nq_gaps = c.nk_gaps = 0;
    const auto gap = [](AttnGaps& g, int& count, int64_t from, int64_t to) {
        if (to > from) {
            g.from[count] = static_cast<int32_t>(from);
            g.to[count++] = static_cast<int32_t>(to);
        }
    };
    for (int32_t i = 0; i < n; ++i) {
        const lora_attn_seq& s = seqs[i];
        if (s.q_rows < 0 || s.k_rows < 0 || s.q_start < q_end || s.k_start < k_end) return LORA_ETABLE;
        // starts first: the sums below then stay inside 64 bits
        if (s.q_start > q_rows || s.k_start > k_rows || s.q_rows > q_rows - s.q_start || s.k_rows > k_rows - s.k_start)
            return LORA_ETABLE;
        gap(c.q_gaps, c.nq_gaps, q_end, s.q_start);
        gap(c.k_gaps, c.nk_gaps, k_end, s.k_start);
        q_end = s.q_start + s.q_rows;
        k_end = s.k_start + s.k_rows;
        if (s.q_rows > 0 || s.k_rows > 0)
            c.order.s[c.n++] = AttnSeq{static_cast<int32_t>(s.q_start), static_cast<int32_t>(s.k_start),
                                       static_cast<int32_t>(s.q_rows), static_cast<int32_t>(s.k_rows), 0, 0, 0};
    }
    gap(c.q_gaps, c.nq_gaps, q_end, q_rows);
    gap(c.k_gaps, c.nk_gaps, k_end, k_rows);
    return LORA_OK;
}

lora_status check_shape(const lora_attn_shape& a, Prepared& c) {
    if (a.q_rows < 0 || a.k_rows < 0 || a.q_rows > LORA_MAX_ROWS || a.k_rows > LORA_MAX_ROWS) return LORA_ESHAPE;
    if (a.q_heads < 1 || a.kv_heads < 1 || a.q_heads > LORA_ATTN_MAX_HEADS || a.q_heads % a.kv_heads) return LORA_ESHAPE;
    if (a.head_dim < 8 || a.head_dim > LORA_ATTN_MAX_HEAD_DIM || a.head_dim % 8) return LORA_ESHAPE;
    if (!(a.scale > 0.f) || !std::isfinite(a.scale)) return LORA_EINVAL;
    AttnShape& s = c.sh;
    std::memset(&s, 0, sizeof(s));
    s.hq = a.q_heads;
    s.hkv = a.kv_heads;
    s.group = a.q_heads / a.kv_heads;
    s.hp = 1;
    while (s.hp < kAttnTile && s.group % (2 * s.hp) == 0) {
        s.hp *= 2;
        ++s.hp_log2;
    }
    s.packs = s.hq / s.hp;
    s.d = a.head_dim;
    s.d16 = (a.head_dim + 15) / 16 * 16;
    s.scale = a.scale;
    s.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    return LORA_OK;
}

lora_status check_workspace(void* ws, size_t have, size_t need) {
    if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 || have < need) return LORA_EWORKSPACE;
    return LORA_OK;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

size_t delta_bytes(int64_t q_rows, int32_t q_heads) {
    return up256(static_cast<size_t>(q_rows) * static_cast<size_t>(q_heads) * 4);
}

int64_t tiles_of(int64_t rows, int per) { return (rows + per - 1) / per; }

// Numbers the items (tiles) of every sequence, in the table's order.
template <class Tiles>
lora_status number_items(Prepared& c, Tiles tiles) {
    int64_t items = 0;
    for (int i = 0; i < c.n; ++i) {
        c.order.s[i].item0 = static_cast<int32_t>(items);
        items += tiles(c.order.s[i]);
        if (items > 0x7FFFFFFF) return LORA_ESHAPE;
    }
    c.sh.n_seqs = c.n;
    c.sh.items = static_cast<int32_t>(items);
    return LORA_OK;
}

void order_by_keys(Prepared& c) {
    std::stable_sort(c.order.s, c.order.s + c.n, [](const AttnSeq& a, const AttnSeq& b) { return a.kl > b.kl; });
}

int key_tiles(const AttnSeq& q) { return static_cast<int>(tiles_of(q.kl, kAttnTile)); }

// Whether the query tiles see at most 512 keys in the mean: the dQ pass then has key tiles of 64 (k_attn_bwd.cu: the two
// forms meet there).
bool few_keys(const Prepared& c, int tokens) {
    int64_t tiles = 0, keys = 0;
    for (int i = 0; i < c.n; ++i) {
        const AttnSeq& q = c.order.s[i];
        const int64_t t = tiles_of(q.ql, tokens);
        tiles += t;
        keys += t * std::max(q.kl - q.ql / 2, q.kl / 2);
    }
    return keys <= 512 * tiles;
}

int q_items(const AttnSeq& q, const AttnShape& sh, int most) {
    int n = attn_query_tiles(q, sh);
    for (int over = most; attn_tiles_seeing(q, sh, over) > 0; over += most) n += attn_tiles_seeing(q, sh, over);
    return n;
}

// Splits the keys of the forward's query tiles, where few rows or heads over long ranges would keep a few SMs busy long after
// the others: an item then has at most two thirds of what an SM gets of the call's work, but no fewer than four key tiles.
// Sequences of one query tile are split from there on, longer ones, which a few long tiles do not hold up as much, from
// four times that.  They come first in the table, as the join wants them.  Returns how many they are, and their query tiles.
// (The slots hold them all on 152 SMs; one that did not fit would stay whole.)
// 24 continuations of 1 to 22 tokens over up to 12000 keys, 32/8 heads of 128: 63 us with the join; pieces of all or half
// an SM's share 71 and 77, none 121.  One token over 4096 keys: 12 us, with at least eight tiles a piece 14.  A prompt of
// 8192 tokens with one head of 128: 25 us and 10 for the join, whole 82; with 8/1 heads, 4096 tokens (1.7 times): 45 and 10,
// whole 48.
int split_keys(Prepared& c, int sms, int32_t* most, int* tiles) {
    AttnSeq* const end = c.order.s + c.n;
    int64_t work = 0;
    for (const AttnSeq* q = c.order.s; q != end; ++q) {
        const int t = attn_query_tiles(*q, c.sh);
        if (t > 0) work += static_cast<int64_t>(attn_seen(*q, c.sh, 0) + attn_seen(*q, c.sh, t - 1)) * t * c.sh.packs;   // twice
    }
    *most = static_cast<int32_t>(std::min<int64_t>(std::max<int64_t>(4, tiles_of(work, 3 * sms)), 1 << 30));
    int64_t slots = 0;
    *tiles = 0;
    for (AttnSeq* q = c.order.s; q != end; ++q) {
        const int t = attn_query_tiles(*q, c.sh);
        if (t == 0 || key_tiles(*q) < (t == 1 ? *most + 1 : 4 * static_cast<int64_t>(*most))) continue;
        const int64_t n = static_cast<int64_t>(t) * attn_pieces(*q, *most);
        if ((slots + n) * c.sh.packs > kAttnMaxSlots) continue;
        q->split = static_cast<int32_t>(slots + 1);
        slots += n;
        *tiles += t;
    }
    return static_cast<int>(std::stable_partition(c.order.s, end, [](const AttnSeq& q) { return q.split != 0; }) - c.order.s);
}

int kv_items(const AttnSeq& q, const AttnShape& sh, int most) {
    int n = key_tiles(q);
    for (int over = most; attn_tiles_over(q, sh, over) > 0; over += most) n += attn_tiles_over(q, sh, over);
    return n;
}

// Splits the queries of dK and dV where a key tile sees more of them than one and a half times what an SM gets of the call's
// work (few key/value heads, shared by many query heads): an item then has that share at most, but no fewer than four
// query tiles.  These sequences come first in the table.  Returns how many they are, and their key tiles.  One sequence of
// 2048 tokens with 8/1 heads of 128: 25 us and 8 for the join, pieces of half that length 33 and 15, none 177; of 4096
// tokens 82 and 6, 74 and 10, 342.  One that does not fit the slots (few queries over many keys: one batch in a thousand of those
// that are split) stays whole, and the others are still looked at: 890 queries over 14344 keys before samples of 1169 and
// 981 with 10/1 heads 117 us and 6, 155 without; where the whole one takes longest all the same, the join's 6 us more.
int split_queries(Prepared& c, int sms, int32_t* most, int* tiles) {
    AttnSeq* const end = c.order.s + c.n;
    int64_t work = 0;
    for (AttnSeq* q = c.order.s; q != end; ++q) {
        q->split = 0;
        const int64_t first = attn_turns(*q, c.sh, 0), last = attn_turns(*q, c.sh, std::max(key_tiles(*q) - 1, 0));
        work += (first + last) * key_tiles(*q) / 2 * c.sh.hkv;   // falling along the keys
    }
    *most = static_cast<int32_t>(std::min<int64_t>(std::max<int64_t>(4, tiles_of(work, sms)), 1 << 30));
    int64_t slots = 0;
    *tiles = 0;
    for (AttnSeq* q = c.order.s; q != end; ++q) {
        if (attn_turns(*q, c.sh, 0) * 2 <= *most * 3) continue;
        const int64_t n = kv_items(*q, c.sh, *most);
        if ((slots + n) * c.sh.hkv > kMaxKvSlots || *tiles + key_tiles(*q) > 65535) continue;
        q->split = static_cast<int32_t>(slots + 1);
        slots += n;
        *tiles += key_tiles(*q);
    }
    return static_cast<int>(std::stable_partition(c.order.s, end, [](const AttnSeq& q) { return q.split != 0; }) - c.order.s);
}

AttnMat mat(const lora_bf16* p, const lora_attn_strides& s) { return AttnMat{const_cast<uint16_t*>(p), s.row, s.head}; }

// Unused rows times heads that an item fills at most, and that an SM's two items of a moment fill at most over the call; a batch
// with more of them gets a kernel for them.  The items write them before their first turn, eight in 0.27 us, the kernel
// costs a launch of some 2 us.  us, by the items and by the kernel, 32/8 heads of 128: one sample of 77 tokens in 128 rows (68 an
// item) 21 and 23; 14 samples of 152 to 1094 tokens on 128-row boundaries (91 of all) both directions 275 and 280; 2000 tokens with
// 512, 1024, 2048 rows after them (54, 108, 216 of all) 43.7, 46.3, 51.8 and 43.2, 45.6, 46.4; 64 samples of 77 tokens every 128
// rows (344 of all) 50 and 45, backward 132 and 121; one token over 300 keys in a buffer of 8192 rows 1116 and 23.
constexpr int64_t kItemFill = 96;

// Gives every unused row of an output with `rows` rows to the items of c (numbered already): the rows after a sequence
// to its own tiles, `tile` rows each, those before the first and after the last to all.  False if the rows need a launch of
// their own.  `heads`: of an item, of `all_heads`; `first` and `len` read a sequence's place.
template <class First, class Len>
bool share_gaps(Prepared& c, const AttnGaps& gaps, int n_gaps, int64_t rows, int tile, int heads, int all_heads, int sms,
                First first, Len len) {
    const auto none = [&c] {
        c.sh.lead = c.sh.trail0 = c.sh.trail = 0;
        for (int i = 0; i < c.n; ++i) c.order.s[i].gap = 0;
        return false;
    };
    none();
    if (n_gaps == 0) return true;
    if (c.sh.items == 0) return false;
    thread_local std::pair<int32_t, int32_t> ends[kAttnMaxSeqs];   // end row, place in the table
    int m = 0;
    for (int i = 0; i < c.n; ++i)
        if (len(c.order.s[i]) > 0) ends[m++] = {first(c.order.s[i]) + len(c.order.s[i]), i};
    std::sort(ends, ends + m);
    int64_t unused = 0;
    for (int g = 0; g < n_gaps; ++g) {
        const int32_t from = gaps.from[g], to = gaps.to[g];
        unused += to - from;
        if (from == 0) {
            c.sh.lead = to;
        } else if (to == rows) {
            c.sh.trail0 = from;
            c.sh.trail = to - from;
        } else {
            const auto e = std::lower_bound(ends, ends + m, std::make_pair(from, int32_t{-1}));
            if (e == ends + m || e->first != from) return none();
            AttnSeq& q = c.order.s[e->second];
            if (static_cast<int64_t>(to - from) * heads > kItemFill * tiles_of(len(q), tile)) return none();
            q.gap = to - from;
        }
    }
    if ((static_cast<int64_t>(c.sh.lead) + c.sh.trail) * heads > kItemFill * c.sh.items) return none();
    if (unused * all_heads > kItemFill * 2 * sms) return none();
    return true;
}

lora_status fill(const AttnGaps& gaps, int n, AttnMat a, AttnMat b, int heads, int d, float* lse, cudaStream_t s) {
    if (n == 0) return LORA_OK;
    AttnFillParams f{a, b, heads, d, lse, n};
    LORA_CUDA(timed(kAttnFill, s, [&] { return launch_attn_fill(f, gaps, s); }));
    return LORA_OK;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

size_t attn_workspace_size(int64_t q_rows, int32_t q_heads) {
    if (q_rows < 0 || q_heads < 0) return 0;
    return kStatusBytes + kSplitBytes + delta_bytes(q_rows, q_heads);
}

lora_status attn_fwd(const lora_bf16* Q, const lora_bf16* K, const lora_bf16* V, const lora_attn_shape* shape,
                     const lora_attn_seq* seqs, int32_t n_seqs, lora_bf16* O, float* lse, void* workspace,
                     size_t workspace_bytes, void* stream) {
    if (!shape) return LORA_EINVAL;
    const lora_attn_shape& a = *shape;
    thread_local Prepared c;   // large: off the stack, one per calling thread
    lora_status st = check_shape(a, c);
    if (st) return st;
    if (a.q_rows > 0 && !lse) return LORA_EINVAL;
    if (!aligned16(lse)) return LORA_EALIGN;
    if ((st = check_mat(Q, a.q, a.q_rows, a.q_heads, a.head_dim))) return st;
    if ((st = check_mat(K, a.k, a.k_rows, a.kv_heads, a.head_dim))) return st;
    if ((st = check_mat(V, a.v, a.k_rows, a.kv_heads, a.head_dim))) return st;
    if ((st = check_mat(O, a.o, a.q_rows, a.q_heads, a.head_dim))) return st;
    if ((st = check_seqs(seqs, n_seqs, a.q_rows, a.k_rows, c))) return st;
    if ((st = check_workspace(workspace, workspace_bytes, kStatusBytes))) return st;
    int sms = 0;
    if ((st = device_setup(&sms))) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    order_by_keys(c);
    const int tokens = kAttnTile / c.sh.hp;
    int32_t most = 0;
    int split_tiles = 0;
    const int split = workspace_bytes >= kStatusBytes + kSplitBytes ? split_keys(c, sms, &most, &split_tiles) : 0;
    if ((st = number_items(c, [&](const AttnSeq& q) { return q.split ? q_items(q, c.sh, most) : attn_query_tiles(q, c.sh); })))
        return st;
    if (!share_gaps(c, c.q_gaps, c.nq_gaps, a.q_rows, tokens, c.sh.hp, a.q_heads, sms, [](const AttnSeq& q) { return q.q0; },
                    [](const AttnSeq& q) { return q.ql; })) {
        if ((st = fill(c.q_gaps, c.nq_gaps, mat(O, a.o), AttnMat{}, a.q_heads, a.head_dim, lse, s))) return st;
    }
    if (c.sh.items == 0) return LORA_OK;
    thread_local AttnFwdParams p;
    std::memset(&p, 0, sizeof(p));
    p.sh = c.sh;
    // no keys at all: the maps describe one row that is never read
    const lora_bf16* k = a.k_rows > 0 ? K : Q;
    const lora_bf16* v = a.k_rows > 0 ? V : Q;
    const int64_t kr = std::max<int64_t>(a.k_rows, 1);
    if (!make_map_heads(&p.mapQ, Q, a.head_dim, a.q_heads, a.q_rows, a.q.head, a.q.row, c.sh.hp, tokens) ||
        !make_map_heads(&p.mapK, k, a.head_dim, a.kv_heads, kr, a.k.head, a.k.row, 1, kAttnTile) ||
        !make_map_heads(&p.mapV, v, a.head_dim, a.kv_heads, kr, a.v.head, a.v.row, 1, kAttnTile))
        return LORA_ECUDA;
    p.O = mat(O, a.o);
    p.lse = lse;
    p.ctl = DevCtl{static_cast<int*>(workspace), wait_limit_ns()};
    p.most = most;
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kStatusBytes);
    LORA_CUDA(timed(kAttnFwd, s, [&] { return launch_attn_fwd(p, c.order, s); }));
    if (split > 0) LORA_CUDA(timed(kAttnJoin, s, [&] { return launch_attn_join(p, c.order, split, split_tiles, s); }));
    return LORA_OK;
}

lora_status attn_bwd(const lora_bf16* dO, const lora_bf16* Q, const lora_bf16* K, const lora_bf16* V,
                     const lora_bf16* O, const float* lse, const lora_attn_shape* shape, const lora_attn_seq* seqs,
                     int32_t n_seqs, lora_bf16* dQ, lora_bf16* dK, lora_bf16* dV, void* workspace,
                     size_t workspace_bytes, void* stream) {
    if (!shape) return LORA_EINVAL;
    const lora_attn_shape& a = *shape;
    thread_local Prepared c;
    lora_status st = check_shape(a, c);
    if (st) return st;
    if (a.q_rows > 0 && !lse) return LORA_EINVAL;
    if (!aligned16(lse)) return LORA_EALIGN;
    if ((st = check_mat(dO, a.d_o, a.q_rows, a.q_heads, a.head_dim))) return st;
    if ((st = check_mat(Q, a.q, a.q_rows, a.q_heads, a.head_dim))) return st;
    if ((st = check_mat(K, a.k, a.k_rows, a.kv_heads, a.head_dim))) return st;
    if ((st = check_mat(V, a.v, a.k_rows, a.kv_heads, a.head_dim))) return st;
    if ((st = check_mat(O, a.o, a.q_rows, a.q_heads, a.head_dim))) return st;
    if ((st = check_mat(dQ, a.d_q, a.q_rows, a.q_heads, a.head_dim))) return st;
    if ((st = check_mat(dK, a.d_k, a.k_rows, a.kv_heads, a.head_dim))) return st;
    if ((st = check_mat(dV, a.d_v, a.k_rows, a.kv_heads, a.head_dim))) return st;
    if ((st = check_seqs(seqs, n_seqs, a.q_rows, a.k_rows, c))) return st;
    if ((st = check_workspace(workspace, workspace_bytes, kStatusBytes + delta_bytes(a.q_rows, a.q_heads)))) return st;
    int sms = 0;
    if ((st = device_setup(&sms))) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const AttnMat mk = mat(dK, a.d_k), mv = mat(dV, a.d_v);
    if (c.n == 0) {
        if ((st = fill(c.q_gaps, c.nq_gaps, mat(dQ, a.d_q), AttnMat{}, a.q_heads, a.head_dim, nullptr, s))) return st;
        return fill(c.k_gaps, c.nk_gaps, mk, mv, a.kv_heads, a.head_dim, nullptr, s);
    }
    order_by_keys(c);
    thread_local AttnBwdParams p;
    std::memset(&p, 0, sizeof(p));
    const int tokens = kAttnTile / c.sh.hp;
    const bool no_q = a.q_rows == 0, no_k = a.k_rows == 0;
    const int64_t qr = std::max<int64_t>(a.q_rows, 1), kr = std::max<int64_t>(a.k_rows, 1);
    const lora_bf16* any = no_q ? K : Q;
    if (!make_map_heads(&p.mapQ, no_q ? any : Q, a.head_dim, a.q_heads, qr, a.q.head, a.q.row, c.sh.hp, tokens) ||
        !make_map_heads(&p.mapO, no_q ? any : O, a.head_dim, a.q_heads, qr, a.o.head, a.o.row, c.sh.hp, tokens) ||
        !make_map_heads(&p.mapDO, no_q ? any : dO, a.head_dim, a.q_heads, qr, a.d_o.head, a.d_o.row, c.sh.hp, tokens))
        return LORA_ECUDA;
    p.lse = lse;
    p.delta = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kStatusBytes);
    p.O = mat(O, a.o);
    p.dQ = mat(dQ, a.d_q);
    p.dK = mk;
    p.dV = mv;
    p.ctl = DevCtl{static_cast<int*>(workspace), wait_limit_ns()};
    if ((st = number_items(c, [&](const AttnSeq& q) { return tiles_of(q.ql, tokens); }))) return st;
    if (!share_gaps(c, c.q_gaps, c.nq_gaps, a.q_rows, tokens, c.sh.hp, a.q_heads, sms, [](const AttnSeq& q) { return q.q0; },
                    [](const AttnSeq& q) { return q.ql; })) {
        if ((st = fill(c.q_gaps, c.nq_gaps, p.dQ, AttnMat{}, a.q_heads, a.head_dim, nullptr, s))) return st;
    }
    p.sh = c.sh;
    const bool short_keys = few_keys(c, tokens);
    const auto key_maps = [&](int rows) {
        return make_map_heads(&p.mapK, no_k ? any : K, a.head_dim, a.kv_heads, kr, a.k.head, a.k.row, 1, rows) &&
               make_map_heads(&p.mapV, no_k ? any : V, a.head_dim, a.kv_heads, kr, a.v.head, a.v.row, 1, rows);
    };
    if (!key_maps(short_keys ? kAttnTile / 2 : kAttnTile)) return LORA_ECUDA;
    if (c.sh.items > 0) LORA_CUDA(timed(kAttnDq, s, [&] { return launch_attn_dq(p, c.order, short_keys, s); }));
    if (short_keys && !key_maps(kAttnTile)) return LORA_ECUDA;
    int split = 0, split_tiles = 0;
    if (workspace_bytes >= kStatusBytes + delta_bytes(a.q_rows, a.q_heads) + kSplitBytes)
        split = split_queries(c, sms, &p.most, &split_tiles);
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kStatusBytes + delta_bytes(a.q_rows, a.q_heads));
    if ((st = number_items(c, [&](const AttnSeq& q) { return q.split ? kv_items(q, c.sh, p.most) : key_tiles(q); })))
        return st;
    if (!share_gaps(c, c.k_gaps, c.nk_gaps, a.k_rows, kAttnTile, 1, a.kv_heads, sms, [](const AttnSeq& q) { return q.k0; },
                    [](const AttnSeq& q) { return q.kl; })) {
        if ((st = fill(c.k_gaps, c.nk_gaps, mk, mv, a.kv_heads, a.head_dim, nullptr, s))) return st;
    }
    p.sh = c.sh;
    if (c.sh.items > 0) LORA_CUDA(timed(kAttnDkDv, s, [&] { return launch_attn_dkdv(p, c.order, s); }));
    if (split > 0) LORA_CUDA(timed(kAttnJoin, s, [&] { return launch_attn_kv_join(p, c.order, split, split_tiles, s); }));
    return LORA_OK;
}

}  // extern "C"
