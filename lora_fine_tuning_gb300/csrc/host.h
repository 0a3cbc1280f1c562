// Host-side helpers shared by the files that implement the C ABI (api.cu defines them).
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda.h>
#include <cuda_runtime.h>

#include "lora.h"

namespace lora {

// True on success; otherwise keeps the error's text for lora_last_error_string().
bool cuda_ok(cudaError_t e);

#define LORA_CUDA(expr)                          \
    do {                                         \
        if (!cuda_ok(expr)) return LORA_ECUDA;   \
    } while (0)

// First use of the current device: checks its architecture and configures every kernel.  *sms: its SM count.
lora_status device_setup(int* sms);

// Limit of the kernels' bounded waits (lora_set_wait_limit_ns).
uint64_t wait_limit_ns();

// Kinds of launches lora_timing_end() reports, in the order of lora_kernel_name().
enum Kind : int {
    kDownProj = 0, kFinalizeS, kGemmFwd, kDsDb, kFinalize, kGemmBwd, kDa, kFinalizeDa, kMemset,
    kDoraU, kDoraNorm, kDoraDz, kDoraDmag,
    kAttnFwd, kAttnJoin, kAttnDq, kAttnDkDv, kAttnFill, kLossRows, kLossPairs, kLossGrad, kLossSum,
    kAdamW, kKinds
};
static_assert(static_cast<int>(kKinds) == static_cast<int>(LORA_KERNEL_KINDS), "the header counts the kinds");

// Runs `launch` (which enqueues work on `s`); when timing is on, brackets it with events.
cudaError_t timed_call(int kind, cudaStream_t s, cudaError_t (*launch)(void*), void* ctx);

template <class F>
cudaError_t timed(int kind, cudaStream_t s, F&& launch) {
    using Fn = typename std::remove_reference<F>::type;
    return timed_call(kind, s, [](void* c) -> cudaError_t { return (*static_cast<Fn*>(c))(); },
                      const_cast<void*>(static_cast<const void*>(&launch)));
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// 3-D bf16 tensor map of `rows` x `heads` x `d` (d contiguous; strides in elements), read in boxes of 64
// features x box_heads x box_rows with the 128-byte swizzle; features past d read as zero.
bool make_map_heads(CUtensorMap* map, const void* base, int d, int heads, int64_t rows, int64_t head_stride,
                    int64_t row_stride, int box_heads, int box_rows);

}  // namespace lora
