// C ABI of the norms around a block: validation, workspace layout and launches.  See include/lora.h for the contract.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "act8.h"
#include "host.h"
#include "norm.h"

namespace lora {
namespace {

constexpr int kMaxSms = 160;   // workspaces are sized without a device; a launch uses as many SMs at most

bool aligned(const void* p, unsigned bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// One matrix of the call: `p` may be null where it is not `needed`.
struct Arguments {
    int64_t rows, width;
    lora_status st = LORA_OK;
    bool vectors = true, ragged = false;
    void fail(lora_status s) {
        if (!st) st = s;
    }
    void matrix(const void* p, int64_t ld, int size, bool needed) {
        if (!p) {
            if (needed && rows > 0) fail(LORA_EINVAL);
            return;
        }
        if (ld < width || ld >= (int64_t{1} << 38)) fail(LORA_ESHAPE);
        if (!aligned(p, size)) fail(LORA_EALIGN);
        ragged = ragged || !aligned16(p) || (ld * size) % 16;
    }
    NormVec vec(const lora_vector& v, bool whole) {
        if (!v.data) return NormVec{nullptr, 0};
        if (v.dtype != LORA_BF16 && v.dtype != LORA_F32) fail(LORA_EINVAL);
        if (!aligned(v.data, v.dtype == LORA_F32 ? 4 : 2)) fail(LORA_EALIGN);
        if (whole) vectors = vectors && aligned16(v.data);
        return NormVec{v.data, v.dtype == LORA_F32};
    }
    NormAct8 act8(const lora_act8* a) {
        if (!a) return NormAct8{nullptr, nullptr};
        if (rows > 0 && (!a->codes || !a->scales)) fail(LORA_EINVAL);
        if (!aligned16(a->codes) || !aligned(a->scales, 4)) fail(LORA_EALIGN);
        return NormAct8{reinterpret_cast<uint8_t*>(a->codes), a->scales};
    }
};

lora_status check_shape(const lora_norm* n, Arguments& c, NormShape& s) {
    if (!n) return LORA_EINVAL;
    if (n->rows < 0 || n->rows > LORA_MAX_ROWS || n->width < 1 || n->width > LORA_MAX_NORM_WIDTH) return LORA_ESHAPE;
    if (n->stream_dtype != LORA_BF16 && n->stream_dtype != LORA_F32) return LORA_EINVAL;
    if (!(n->eps >= 1e-30f) || !std::isfinite(n->eps) || !std::isfinite(n->w_offset) || !std::isfinite(n->res_scale)) return LORA_EINVAL;
    c.rows = n->rows;
    c.width = n->width;
    c.vectors = n->width % 8 == 0;
    c.ragged = !c.vectors;
    s.rows = static_cast<int32_t>(n->rows);
    s.width = static_cast<int32_t>(n->width);
    s.f32 = n->stream_dtype == LORA_F32;
    s.w = c.vec(n->w, true);
    s.post = c.vec(n->post_w, true);
    s.gate = c.vec(n->gate, true);
    s.row_gate = c.vec(n->row_gate, false);
    s.eps = n->eps;
    s.offset = n->w_offset;
    s.res = n->res_scale;
    s.vectors = c.vectors;
    s.inv_width = static_cast<float>(1.0 / static_cast<double>(n->width));
    s.codes_ld = act8_codes_ld(n->width);
    s.scales_ld = act8_scales_ld(n->width);
    return c.st;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

size_t norm_workspace_size(int64_t rows, int64_t width) {
    if (rows < 0 || rows > LORA_MAX_ROWS || width < 1 || width > LORA_MAX_NORM_WIDTH) return 0;
    const int groups = norm_bwd_groups(static_cast<int>(std::max<int64_t>(rows, 1)), static_cast<int>(width), kMaxSms);
    return 256 + (static_cast<size_t>(groups) * 2 * static_cast<size_t>(width) * 4 + 255) / 256 * 256;
}

lora_status norm_fwd(const lora_norm* norm, const void* h, const lora_bf16* y, void* h_out, lora_bf16* x,
                     const lora_act8* x8, const lora_act8* h8, const lora_act8* y8, void* stream) {
    NormFwd p;
    std::memset(&p, 0, sizeof(p));
    Arguments c{};
    lora_status st = check_shape(norm, c, p.s);
    if (st) return st;
    const int size = p.s.f32 ? 4 : 2;
    const bool has_w = norm->w.data != nullptr;
    // without a block's output nothing is added, and the stream stays where it is
    // (an empty tensor's address may be null: what a call leaves out is told apart where there are rows)
    const bool rows = norm->rows > 0;
    if (rows && !y && (norm->post_w.data || norm->gate.data || norm->row_gate.data || h_out || y8)) return LORA_EINVAL;
    if (!has_w && rows && (x || x8 || !y)) return LORA_EINVAL;
    if (has_w && rows && !x && !x8) return LORA_EINVAL;
    c.matrix(h, norm->h, size, true);
    c.matrix(y, norm->y, 2, false);
    c.matrix(h_out, norm->h_out, size, y != nullptr);
    c.matrix(x, norm->x, 2, false);
    p.x8 = c.act8(x8);
    p.h8 = c.act8(h8);
    p.y8 = c.act8(y8);
    if (c.st) return c.st;
    if (h_out == h && y && norm->rows > 1 && norm->h_out != norm->h) return LORA_EINVAL;   // in place: written where it was read
    int sms = 0;
    if ((st = device_setup(&sms))) return st;
    if (norm->rows == 0) return LORA_OK;
    p.s.ragged = c.ragged;
    p.h = h, p.y = y, p.h_out = h_out, p.x = x;
    p.h_ld = norm->h * size, p.y_ld = norm->y * 2, p.h_out_ld = norm->h_out * size, p.x_ld = norm->x * 2;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LORA_CUDA(timed(kNormFwd, s, [&] { return launch_norm_fwd(p, sms, s); }));
    return LORA_OK;
}

lora_status norm_bwd(const lora_norm* norm, const lora_bf16* dx, const void* dh, const void* h, const lora_act8* h8,
                     const lora_bf16* y, const lora_act8* y8, void* dh_out, lora_bf16* dy, float* dw, float* dpost_w,
                     float* dgate, float* drow_gate, void* workspace, size_t workspace_bytes, void* stream) {
    NormBwd p;
    std::memset(&p, 0, sizeof(p));
    Arguments c{};
    lora_status st = check_shape(norm, c, p.s);
    if (st) return st;
    const int size = p.s.f32 ? 4 : 2;
    const bool has_w = norm->w.data != nullptr, has_y = y || y8;
    if ((h && h8) || (y && y8)) return LORA_EINVAL;
    const bool rows = norm->rows > 0;
    if (rows && !has_y && (norm->post_w.data || norm->gate.data || norm->row_gate.data || dy)) return LORA_EINVAL;
    if (!has_w && (dw || (rows && (dx || h || h8 || !has_y)))) return LORA_EINVAL;
    if ((dpost_w && !norm->post_w.data) || (dgate && !norm->gate.data) || (drow_gate && !norm->row_gate.data)) return LORA_EINVAL;
    c.matrix(dx, norm->dx, 2, has_w);
    c.matrix(dh, norm->dh, size, false);
    c.matrix(h, norm->h, size, has_w && !h8);
    c.matrix(y, norm->y, 2, false);
    c.matrix(dh_out, norm->dh_out, size, true);
    c.matrix(dy, norm->dy, 2, false);
    p.h8 = c.act8(h8);
    p.y8 = c.act8(y8);
    if (c.st) return c.st;
    if ((dh_out == dh && norm->rows > 1 && norm->dh_out != norm->dh) || (dy && (dy == dh_out || dy == dh))) return LORA_EINVAL;
    if (!aligned(dw, 4) || !aligned(dpost_w, 4) || !aligned(dgate, 4) || !aligned(drow_gate, 4)) return LORA_EALIGN;
    const bool sums = dw || dpost_w || dgate;
    if (sums && (!workspace || !aligned(workspace, 256) || workspace_bytes < norm_workspace_size(norm->rows, norm->width)))
        return LORA_EWORKSPACE;
    int sms = 0;
    if ((st = device_setup(&sms))) return st;
    sms = std::min(sms, kMaxSms);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    p.dx = dx, p.dh = dh, p.h = h, p.y = y, p.dh_out = dh_out, p.dy = dy;
    p.s.ragged = c.ragged;
    // (a matrix that is not given has no stride: nothing of its rows is shifted)
    const auto bytes = [](const void* q, int64_t ld, int of) { return q ? ld * of : int64_t{0}; };
    p.dx_ld = bytes(dx, norm->dx, 2), p.dh_ld = bytes(dh, norm->dh, size), p.h_ld = bytes(h, norm->h, size), p.y_ld = bytes(y, norm->y, 2);
    p.dh_out_ld = norm->dh_out * size, p.dy_ld = bytes(dy, norm->dy, 2);
    p.dw = dw, p.dpost = dpost_w, p.dgate = dgate, p.drow = drow_gate;
    p.part = sums ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + 256) : nullptr;
    auto* launch = h8 || y8 ? (sums ? launch_norm_bwd8_sums : launch_norm_bwd8) : (sums ? launch_norm_bwd_sums : launch_norm_bwd);
    if (norm->rows > 0) LORA_CUDA(timed(kNormBwd, s, [&] { return launch(p, sms, s); }));
    if (sums) LORA_CUDA(timed(kNormSums, s, [&] { return launch_norm_sums(p, s); }));
    return LORA_OK;
}

}  // extern "C"
