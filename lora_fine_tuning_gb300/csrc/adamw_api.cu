// C ABI of the AdamW step: validation and launches.  See include/lora.h for the contract.
#include <cmath>
#include <cstring>

#include "adamw.h"
#include "host.h"

namespace lora {
namespace {

lora_status check_tensor(const lora_adamw_tensor& t) {
    if (t.n < 0 || t.n > (int64_t{1} << 40)) return LORA_ESHAPE;
    if (t.n == 0) return LORA_OK;
    if (!t.param || !t.grad || !t.m || !t.v) return LORA_EINVAL;
    if ((t.param_dtype != LORA_BF16 && t.param_dtype != LORA_F32) || (t.grad_dtype != LORA_BF16 && t.grad_dtype != LORA_F32))
        return LORA_EINVAL;
    if (t.state_bits != 8 && t.state_bits != 32) return LORA_EINVAL;
    if (t.state_bits == 8 && (!t.m_scale || !t.v_scale)) return LORA_EINVAL;
    if (t.master && t.param_dtype == LORA_F32) return LORA_EINVAL;
    if (!aligned16(t.param) || !aligned16(t.grad) || !aligned16(t.m) || !aligned16(t.v) || !aligned16(t.master))
        return LORA_EALIGN;
    if (reinterpret_cast<uintptr_t>(t.m_scale) % 4 || reinterpret_cast<uintptr_t>(t.v_scale) % 4) return LORA_EALIGN;
    return LORA_OK;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

lora_status adamw_step(const lora_adamw_tensor* tensors, int32_t n_tensors, double lr, double beta1, double beta2,
                       double eps, double weight_decay, int64_t step, const float* grad_scale, void* stream) {
    if (n_tensors < 0 || (n_tensors > 0 && !tensors)) return LORA_EINVAL;
    if (!std::isfinite(lr) || !std::isfinite(weight_decay) || !(eps >= 1e-30) || !std::isfinite(static_cast<float>(eps))) return LORA_EINVAL;
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || step < 1) return LORA_EINVAL;
    if (reinterpret_cast<uintptr_t>(grad_scale) % 4) return LORA_EALIGN;
    for (int32_t i = 0; i < n_tensors; ++i) {
        const lora_status st = check_tensor(tensors[i]);
        if (st) return st;
    }
    int sms = 0;
    const lora_status st = device_setup(&sms);
    if (st) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    AdamStep p;
    p.b1 = static_cast<float>(beta1);
    p.b1c = static_cast<float>(1.0 - beta1);
    p.b2 = static_cast<float>(beta2);
    p.b2c = static_cast<float>(1.0 - beta2);
    p.keep = static_cast<float>(1.0 - lr * weight_decay);
    p.rate = static_cast<float>(-lr / (1.0 - std::pow(beta1, static_cast<double>(step))));
    p.inv_c2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, static_cast<double>(step))));
    p.eps = static_cast<float>(eps);
    p.one = 1.f;
    p.grad_scale = grad_scale;
    thread_local AdamTensors<kAdamTensors> table;
    // the tensors with fp32 states, then those with 8-bit ones: a launch for every kAdamTensors of a kind
    for (const int bits : {32, 8}) {
        const int64_t each = bits == 8 ? kAdamChunk8 : kAdamChunk32;
        int64_t chunks = 0;
        p.n = 0;
        const auto flush = [&]() -> lora_status {
            if (p.n == 0) return LORA_OK;
            LORA_CUDA(timed(kAdamW, s, [&] { return launch_adamw(p, table, bits == 8, static_cast<int>(chunks), s); }));
            p.n = 0;
            chunks = 0;
            return LORA_OK;
        };
        for (int32_t i = 0; i < n_tensors; ++i) {
            const lora_adamw_tensor& t = tensors[i];
            if (t.n == 0 || t.state_bits != bits) continue;
            const int64_t c = (t.n + each - 1) / each;   // at most 2^29: a launch's count stays below 2^31
            if (p.n == kAdamTensors || chunks + c > (int64_t{1} << 30)) {
                const lora_status f = flush();
                if (f) return f;
            }
            table.chunk0[p.n] = static_cast<int32_t>(chunks);
            table.t[p.n++] = AdamTensor{t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.master, t.n,
                                        (t.param_dtype == LORA_F32 ? kAdamParamF32 : 0u) |
                                            (t.grad_dtype == LORA_F32 ? kAdamGradF32 : 0u)};
            chunks += c;
        }
        const lora_status f = flush();
        if (f) return f;
    }
    return LORA_OK;
}

}  // extern "C"
