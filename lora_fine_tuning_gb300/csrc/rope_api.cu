// C ABI of the rotary positions: the table of frequencies, validation and launches.  See include/lora.h for the contract.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "host.h"
#include "rope.h"

namespace lora {
namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

// f / 2 pi modulo one, rounded to 2^-64, of the double f >= 0: its 53-bit fraction times 1 / 2 pi to 128 bits.
uint64_t turns_of(double f) {
    if (!(f > 0)) return 0;
    int e;
    const uint64_t m = static_cast<uint64_t>(std::ldexp(std::frexp(f, &e), 53));   // f = m 2^(e - 53)
    // 1 / 2 pi = 0.159154943091895335768883763372514362... in units of 2^-128
    const unsigned __int128 inv = (static_cast<unsigned __int128>(0x28BE60DB9391054Aull) << 64) | 0x7F09D5F47D4D3770ull;
    // m inv has up to 179 bits: three words, low first
    const unsigned __int128 lo = static_cast<unsigned __int128>(m) * static_cast<uint64_t>(inv);
    const unsigned __int128 hi = static_cast<unsigned __int128>(m) * static_cast<uint64_t>(inv >> 64) + (lo >> 64);
    const uint64_t w[4] = {static_cast<uint64_t>(lo), static_cast<uint64_t>(hi), static_cast<uint64_t>(hi >> 64), 0};
    // turns = (m inv) 2^(e - 53 - 128): bits from 2^-64 on, rounded to nearest
    const int shift = 53 + 128 - 64 - e;   // the place of the bit that counts 2^-64
    const auto bits = [&w](int from) -> uint64_t {
        if (from >= 192) return 0;
        if (from < 0) return from <= -64 ? 0 : w[0] << -from;   // a frequency so large that its turns are whole ones
        const int i = from / 64, s = from % 64;
        return s ? (w[i] >> s) | (w[i + 1] << (64 - s)) : w[i];
    };
    const uint64_t half = shift >= 1 && shift <= 192 ? bits(shift - 1) & 1u : 0u;
    return bits(shift) + half;
}

lora_status check_mat(const void* p, const lora_attn_strides& s, int64_t rows, int heads, int d) {
    if (rows > 0 && heads > 0 && !p) return LORA_EINVAL;
    if (reinterpret_cast<uintptr_t>(p) % 2) return LORA_EALIGN;
    if (heads == 0) return LORA_OK;
    if (s.row < 0 || s.head < 0 || s.row >= (int64_t{1} << 38) || s.head >= (int64_t{1} << 38)) return LORA_ESHAPE;
    // rows of heads, or heads of rows; either way no element twice
    const bool by_row = (heads == 1 || s.head >= d) && (rows <= 1 || s.row >= (heads - 1) * (heads == 1 ? 0 : s.head) + d);
    const bool by_head = (rows <= 1 || s.row >= d) && (heads == 1 || s.head >= (rows - 1) * s.row + d);
    return by_row || by_head ? LORA_OK : LORA_ESHAPE;
}

// In place: every element is written where it was read.
bool same_place(const void* in, const lora_attn_strides& i, const void* out, const lora_attn_strides& o, int64_t rows, int heads) {
    return in != out || ((rows <= 1 || i.row == o.row) && (heads <= 1 || i.head == o.head));
}

// The widest vector (values) that divides everything of `m` it would be used on.
int vector_of(int W, const void* p, const lora_attn_strides& s, int64_t rows, int heads) {
    if (heads == 0) return W;
    while (W > 1 && (reinterpret_cast<uintptr_t>(p) % (2 * W) || (rows > 1 && s.row % W) || (heads > 1 && s.head % W))) W /= 2;
    return W;
}

lora_status run(const lora_bf16* Q, const lora_bf16* K, const lora_bf16* V, const void* positions, const int64_t* slots,
                const lora_rope_shape* shape, const lora_rope* rope, lora_bf16* Qo, lora_bf16* Ko, lora_bf16* Vo,
                bool back, bool append, void* stream) {
    if (!shape || !rope) return LORA_EINVAL;
    const lora_rope_shape& g = *shape;
    if (g.rows < 0 || g.rows > LORA_MAX_ROWS) return LORA_ESHAPE;
    if (g.q_heads < 0 || g.kv_heads < 0 || g.q_heads + static_cast<int64_t>(g.kv_heads) < 1 || g.q_heads > LORA_ATTN_MAX_HEADS ||
        g.kv_heads > LORA_ATTN_MAX_HEADS)
        return LORA_ESHAPE;
    if (g.head_dim < 1 || g.head_dim > LORA_ROPE_MAX_HEAD_DIM) return LORA_ESHAPE;
    if (rope->rot_dim < 2 || rope->rot_dim % 2 || rope->rot_dim > g.head_dim) return LORA_ESHAPE;
    if ((rope->interleaved != 0 && rope->interleaved != 1) || !std::isfinite(rope->magnitude)) return LORA_EINVAL;
    if (g.positions_bits != 64 && g.positions_bits != 32) return LORA_EINVAL;
    if (g.rows > 0 && (!positions || (append && !slots))) return LORA_EINVAL;
    if (reinterpret_cast<uintptr_t>(positions) % (g.positions_bits / 8) || reinterpret_cast<uintptr_t>(slots) % 8) return LORA_EALIGN;
    if (append && (g.kv_heads < 1 || g.cache_rows < 0 || g.cache_rows >= (int64_t{1} << 38))) return LORA_ESHAPE;
    const int d = g.head_dim, hq = g.q_heads, hk = g.kv_heads;
    const int64_t out_rows = append ? g.cache_rows : g.rows;
    lora_status st;
    if ((st = check_mat(Q, g.q, g.rows, hq, d)) || (st = check_mat(K, g.k, g.rows, hk, d)) ||
        (st = check_mat(Qo, g.q_out, g.rows, hq, d)) || (st = check_mat(Ko, g.k_out, out_rows, hk, d)))
        return st;
    if (append && ((st = check_mat(V, g.v, g.rows, hk, d)) || (st = check_mat(Vo, g.v_out, out_rows, hk, d)))) return st;
    if (!same_place(Q, g.q, Qo, g.q_out, g.rows, hq)) return LORA_EINVAL;
    if (append ? (g.rows > 0 && g.cache_rows > 0 && (Ko == K || Vo == V || Ko == Vo))
               : !same_place(K, g.k, Ko, g.k_out, g.rows, hk))
        return LORA_EINVAL;
    int sms = 0;
    if ((st = device_setup(&sms))) return st;
    if (g.rows == 0) return LORA_OK;

    const int rot = rope->rot_dim;
    int W = 8;
    while (W > 1 && ((rot / 2) % W || (d - rot) % W)) W /= 2;
    W = vector_of(W, Q, g.q, g.rows, hq);
    W = vector_of(W, Qo, g.q_out, g.rows, hq);
    W = vector_of(W, K, g.k, g.rows, hk);
    W = vector_of(W, Ko, g.k_out, out_rows, hk);
    if (append) {
        W = vector_of(W, V, g.v, g.rows, hk);
        W = vector_of(W, Vo, g.v_out, out_rows, hk);
    }
    const auto mat = [](const lora_bf16* p, const lora_attn_strides& s) { return RopeMat{const_cast<uint16_t*>(p), s.row, s.head}; };
    RopeParams p;
    std::memset(&p, 0, sizeof(p));
    p.q = mat(Q, g.q), p.k = mat(K, g.k), p.qo = mat(Qo, g.q_out), p.ko = mat(Ko, g.k_out);
    if (append) p.v = mat(V, g.v), p.vo = mat(Vo, g.v_out);
    p.rows = static_cast<int32_t>(g.rows), p.q_heads = hq, p.kv_heads = hk, p.d = d, p.rot = rot;
    p.interleaved = rope->interleaved;
    p.back = back;
    // a unit is two vectors
    p.units = rot / 2 / W;
    p.q_copies = Qo != Q ? ((d - rot) / W + 1) / 2 : 0;
    p.k_copies = Ko != K ? ((d - rot) / W + 1) / 2 : 0;
    p.v_units = append ? (d / W + 1) / 2 : 0;
    p.each = std::max({hq ? p.units + p.q_copies : 0, hk ? p.units + p.k_copies : 0, p.v_units});
    p.g = std::max(1, 32 / p.each);
    // an item has as many heads as its lanes take; fewer where the rows would give an SM fewer than sixteen items
    const auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const int64_t least = std::max<int64_t>({1, up(hq, kRopeQHeads * p.g), up(hk, kRopeKHeads * p.g)}), most = std::max<int64_t>(least, up(std::max(hq, hk), p.g));
    p.items = static_cast<int32_t>(std::min(std::max(least, up(static_cast<int64_t>(sms) * 16, g.rows)), most));
    p.q_each = static_cast<int32_t>(up(hq, p.items));
    p.k_each = static_cast<int32_t>(up(hk, p.items));
    p.positions = positions;
    p.positions64 = g.positions_bits == 64;
    p.slots = append ? slots : nullptr;
    p.slot_rows = g.cache_rows;
    p.magnitude = rope->magnitude;
    std::memcpy(p.turn, rope->turn, sizeof(uint64_t) * (rot / 2));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LORA_CUDA(timed(append ? kRopeAppend : kRope, s, [&] { return launch_rope(p, W, sms, s); }));
    return LORA_OK;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

lora_status rope_table(int32_t rot_dim, double base, int32_t interleaved, const lora_rope_scaling* scaling, lora_rope* out) {
    if (!out) return LORA_EINVAL;
    if (rot_dim < 2 || rot_dim % 2 || rot_dim > LORA_ROPE_MAX_HEAD_DIM) return LORA_ESHAPE;
    if (!(base > 0) || !std::isfinite(base) || (interleaved != 0 && interleaved != 1)) return LORA_EINVAL;
    lora_rope_scaling s = {LORA_ROPE_NONE, 1.f, 1.0, 0.0, 0.0, 0.0};
    if (scaling) s = *scaling;
    if (s.kind < LORA_ROPE_NONE || s.kind > LORA_ROPE_PARTS || !std::isfinite(s.magnitude)) return LORA_EINVAL;
    if (s.kind != LORA_ROPE_NONE && (!(s.factor > 0) || !std::isfinite(s.factor))) return LORA_EINVAL;
    if (s.kind == LORA_ROPE_PARTS && (!(s.original > 0) || !std::isfinite(s.original) || !(s.high > s.low) || !std::isfinite(s.high - s.low)))
        return LORA_EINVAL;
    std::memset(out, 0, sizeof(*out));
    out->rot_dim = rot_dim;
    out->interleaved = interleaved;
    out->magnitude = s.magnitude;
    if (s.kind == LORA_ROPE_BASE && rot_dim > 2) base *= std::pow(s.factor, static_cast<double>(rot_dim) / (rot_dim - 2));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (s.kind == LORA_ROPE_LINEAR) f /= s.factor;
        if (s.kind == LORA_ROPE_PARTS) {
            const double keep = std::min(1.0, std::max(0.0, (s.original * f / kTwoPi - s.low) / (s.high - s.low)));
            f = f * keep + f / s.factor * (1.0 - keep);
        }
        if (!std::isfinite(f)) return LORA_EINVAL;
        out->turn[i] = turns_of(f);
    }
    return LORA_OK;
}

lora_status rope_fwd(const lora_bf16* Q, const lora_bf16* K, const void* positions, const lora_rope_shape* shape,
                     const lora_rope* rope, lora_bf16* Q_out, lora_bf16* K_out, void* stream) {
    return run(Q, K, nullptr, positions, nullptr, shape, rope, Q_out, K_out, nullptr, false, false, stream);
}

lora_status rope_bwd(const lora_bf16* dQ, const lora_bf16* dK, const void* positions, const lora_rope_shape* shape,
                     const lora_rope* rope, lora_bf16* dQ_out, lora_bf16* dK_out, void* stream) {
    return run(dQ, dK, nullptr, positions, nullptr, shape, rope, dQ_out, dK_out, nullptr, true, false, stream);
}

lora_status rope_append(const lora_bf16* Q, const lora_bf16* K, const lora_bf16* V, const void* positions,
                        const int64_t* slots, const lora_rope_shape* shape, const lora_rope* rope, lora_bf16* Q_out,
                        lora_bf16* K_cache, lora_bf16* V_cache, void* stream) {
    return run(Q, K, V, positions, slots, shape, rope, Q_out, K_cache, V_cache, false, true, stream);
}

}  // extern "C"
