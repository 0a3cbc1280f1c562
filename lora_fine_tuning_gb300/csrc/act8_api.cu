// C ABI of the activations in 8 bits: validation and launches.  See include/lora.h for the contract.
#include "act8.h"
#include "host.h"

namespace lora {
namespace {

lora_status check(const void* x, int64_t rows, int64_t width, int64_t ld, const lora_act8* a, Act8Params& p) {
    if (!a) return LORA_EINVAL;
    if (rows < 0 || rows > LORA_MAX_ROWS || width < 1 || width > LORA_MAX_ACT8_WIDTH) return LORA_ESHAPE;
    if (ld < width || ld >= (int64_t{1} << 38)) return LORA_ESHAPE;
    const int64_t per_row = act8_codes_ld(width) / 8;
    if (rows * per_row >= (int64_t{1} << 31)) return LORA_ESHAPE;
    if (rows > 0 && (!x || !a->codes || !a->scales)) return LORA_EINVAL;
    if (reinterpret_cast<uintptr_t>(x) % 2 || !aligned16(a->codes) || reinterpret_cast<uintptr_t>(a->scales) % 4) return LORA_EALIGN;
    p = Act8Params{const_cast<uint16_t*>(static_cast<const uint16_t*>(x)), reinterpret_cast<uint8_t*>(a->codes), a->scales,
                   ld, static_cast<int32_t>(width), static_cast<uint32_t>(per_row),
                   static_cast<uint32_t>(rows * per_row), aligned16(x) && ld % 8 == 0, 0, 0};
    // 2^shift < per_row <= 2^(shift + 1): magic = ceil(2^(32 + shift) / per_row) is below 2^32 and exceeds that quotient by less than one,
    // so u magic exceeds u 2^(32 + shift) / per_row by less than 2^31, and the quotient's fraction is at most 1 - 1 / per_row
    while ((uint64_t{2} << p.shift) < static_cast<uint64_t>(per_row)) ++p.shift;
    p.magic = static_cast<uint32_t>(((uint64_t{1} << (32 + p.shift)) + per_row - 1) / per_row);
    return LORA_OK;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

lora_status act8_store(const lora_bf16* X, int64_t rows, int64_t width, int64_t ld, const lora_act8* out, void* stream) {
    Act8Params p;
    lora_status st = check(X, rows, width, ld, out, p);
    if (st) return st;
    int sms = 0;
    if ((st = device_setup(&sms))) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows > 0) LORA_CUDA(timed(kAct8Store, s, [&] { return launch_act8_store(p, s); }));
    return LORA_OK;
}

lora_status act8_load(const lora_act8* in, int64_t rows, int64_t width, lora_bf16* X, int64_t ld, void* stream) {
    Act8Params p;
    lora_status st = check(X, rows, width, ld, in, p);
    if (st) return st;
    int sms = 0;
    if ((st = device_setup(&sms))) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows > 0) LORA_CUDA(timed(kAct8Load, s, [&] { return launch_act8_load(p, s); }));
    return LORA_OK;
}

}  // extern "C"
