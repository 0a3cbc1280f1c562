// C ABI of the losses on logits: validation, workspace layout and launches.  See include/lora.h for the contract.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "host.h"
#include "loss.h"

namespace lora {
namespace {

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

bool aligned(const void* p, unsigned bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

lora_status check_logits(const lora_logits* g, LossLogits& in) {
    if (!g) return LORA_EINVAL;
    if (g->dtype != LORA_BF16 && g->dtype != LORA_F32) return LORA_EINVAL;
    if (g->rows < 0 || g->rows > LORA_MAX_ROWS || g->vocab < 1 || g->vocab > LORA_MAX_VOCAB) return LORA_ESHAPE;
    if (g->ld < g->vocab || g->ld >= (int64_t{1} << 38)) return LORA_ESHAPE;
    if (g->dlogits && (g->dlogits_ld < g->vocab || g->dlogits_ld >= (int64_t{1} << 38))) return LORA_ESHAPE;
    // in place: every element is written where it was read
    if (g->dlogits == g->logits && g->rows > 0 && g->dlogits_ld != g->ld) return LORA_EINVAL;
    if (g->rows > 0 && (!g->logits || !g->labels || !g->logp)) return LORA_EINVAL;
    const int size = g->dtype == LORA_F32 ? 4 : 2;
    if (!aligned(g->logits, size) || !aligned(g->dlogits, size) || !aligned(g->labels, 8) || !aligned(g->logp, 4))
        return LORA_EALIGN;
    in = LossLogits{g->logits, g->dlogits, g->rows, g->ld, g->dlogits_ld, static_cast<int32_t>(g->vocab),
                    g->dtype == LORA_F32 ? 1 : 0, g->labels, g->logp};
    return LORA_OK;
}

struct LossLayout {
    size_t row, coef, pairs, total;
};

LossLayout loss_layout(int64_t rows) {
    LossLayout L;
    L.row = 256;   // after the device status word and the pairs' ticket
    L.coef = L.row + up256(static_cast<size_t>(rows) * sizeof(LossRow));
    L.pairs = L.coef + up256(static_cast<size_t>(rows) * 4);
    L.total = L.pairs + LORA_MAX_PAIRS * 4;
    return L;
}

lora_status check_workspace(void* ws, size_t have, size_t need) {
    if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 || have < need) return LORA_EWORKSPACE;
    return LORA_OK;
}

// Every row belongs to one response at most.
lora_status check_pairs(const lora_pref_pair* pairs, int32_t n, int64_t rows, PrefPairs<kLossMaxPairs>& out) {
    if (n < 0 || n > LORA_MAX_PAIRS) return LORA_ETABLE;
    if (n > 0 && !pairs) return LORA_EINVAL;
    struct Span {
        int64_t from, to;
    };
    thread_local Span spans[2 * kLossMaxPairs];
    int m = 0;
    for (int32_t i = 0; i < n; ++i) {
        const lora_pref_pair& q = pairs[i];
        const int64_t start[2] = {q.chosen_start, q.rejected_start}, len[2] = {q.chosen_rows, q.rejected_rows};
        for (int s = 0; s < 2; ++s) {
            if (start[s] < 0 || len[s] < 0 || start[s] > rows || len[s] > rows - start[s]) return LORA_ETABLE;
            if (len[s] > 0) spans[m++] = Span{start[s], start[s] + len[s]};
        }
        out.p[i] = PrefPair{static_cast<int32_t>(start[0]), static_cast<int32_t>(start[1]), static_cast<int32_t>(len[0]),
                            static_cast<int32_t>(len[1])};
    }
    std::sort(spans, spans + m, [](const Span& a, const Span& b) { return a.from < b.from; });
    for (int i = 1; i < m; ++i)
        if (spans[i].from < spans[i - 1].to) return LORA_ETABLE;
    return LORA_OK;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

size_t loss_workspace_size(int64_t rows) { return rows >= 0 ? loss_layout(rows).total : 0; }

lora_status pref_loss(const lora_logits* logits, const lora_pref_pair* pairs, int32_t n_pairs, const float* ref_logp,
                      float beta, float label_smoothing, float scale, float* loss, float* margins, void* workspace,
                      size_t workspace_bytes, void* stream) {
    thread_local PrefParams p;
    thread_local PrefPairs<kLossMaxPairs> table;
    std::memset(&p, 0, sizeof(p));
    lora_status st = check_logits(logits, p.in);
    if (st) return st;
    if (!loss || (n_pairs > 0 && !margins)) return LORA_EINVAL;
    if (!std::isfinite(beta) || !std::isfinite(scale) || !(label_smoothing >= 0.f && label_smoothing <= 1.f))
        return LORA_EINVAL;
    if (!aligned(ref_logp, 4) || !aligned(loss, 4) || !aligned(margins, 4)) return LORA_EALIGN;
    if ((st = check_pairs(pairs, n_pairs, p.in.rows, table))) return st;
    const LossLayout L = loss_layout(p.in.rows);
    if ((st = check_workspace(workspace, workspace_bytes, loss_workspace_size(p.in.rows)))) return st;
    int sms = 0;
    if ((st = device_setup(&sms))) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.ref = ref_logp;
    p.row = reinterpret_cast<LossRow*>(ws + L.row);
    p.coef = reinterpret_cast<float*>(ws + L.coef);
    p.loss = loss;
    p.margin = margins;
    p.pair_loss = reinterpret_cast<float*>(ws + L.pairs);
    p.ticket = reinterpret_cast<uint32_t*>(ws + 128);   // beside the status word
    p.n_pairs = n_pairs;
    p.beta = beta;
    p.smoothing = label_smoothing;
    p.scale = scale;
    p.ctl = DevCtl{static_cast<int*>(workspace), wait_limit_ns()};
    bool paired = false;
    if (p.in.rows > 0) LORA_CUDA(timed(kLossRows, s, [&] { return launch_loss_stats(p, table, sms, &paired, s); }));
    if (!paired) LORA_CUDA(timed(kLossPairs, s, [&] { return launch_loss_pairs(p, table, s); }));
    if (p.in.rows > 0 && p.in.dz) LORA_CUDA(timed(kLossGrad, s, [&] { return launch_loss_grad(p, s); }));
    return LORA_OK;
}

lora_status policy_loss(const lora_logits* logits, const float* old_logp, const float* advantages,
                        const float* ref_logp, float clip_low, float clip_high, float kl_coef, float scale, float* loss,
                        void* workspace, size_t workspace_bytes, void* stream) {
    PolicyParams p;
    std::memset(&p, 0, sizeof(p));
    lora_status st = check_logits(logits, p.in);
    if (st) return st;
    if (!loss || (p.in.rows > 0 && (!old_logp || !advantages))) return LORA_EINVAL;
    if (!(clip_low >= 0.f && clip_low <= 1.f) || !(clip_high >= 0.f) || !std::isfinite(clip_high)) return LORA_EINVAL;
    if (!std::isfinite(kl_coef) || !std::isfinite(scale)) return LORA_EINVAL;
    if (kl_coef != 0.f && !ref_logp && p.in.rows > 0) return LORA_EINVAL;
    if (!aligned(old_logp, 4) || !aligned(advantages, 4) || !aligned(ref_logp, 4) || !aligned(loss, 4)) return LORA_EALIGN;
    if ((st = check_workspace(workspace, workspace_bytes, loss_workspace_size(p.in.rows)))) return st;
    int sms = 0;
    if ((st = device_setup(&sms))) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    p.old_logp = old_logp;
    p.adv = advantages;
    p.ref = kl_coef != 0.f ? ref_logp : nullptr;
    p.row_loss = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + loss_layout(p.in.rows).row);
    p.ticket = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + 128);   // beside the status word
    p.ctl = DevCtl{static_cast<int*>(workspace), wait_limit_ns()};
    p.loss = loss;
    p.lo = static_cast<float>(1.0 - static_cast<double>(clip_low));
    p.hi = static_cast<float>(1.0 + static_cast<double>(clip_high));
    p.kl = kl_coef;
    p.scale = scale;
    bool summed = false;
    if (p.in.rows > 0) LORA_CUDA(timed(kLossRows, s, [&] { return launch_policy_rows(p, sms, &summed, s); }));
    if (!summed) LORA_CUDA(timed(kLossSum, s, [&] { return launch_loss_sum(p.row_loss, p.in.rows, scale, loss, s); }));
    return LORA_OK;
}

}  // extern "C"
