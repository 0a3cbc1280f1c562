// Launch plan of the rotary positions (k_rope.cu), filled by rope_api.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace lora {

constexpr int kRopeMaxPairs = 128;   // head_dim <= 256
constexpr int kRopeQHeads = 4, kRopeKHeads = 2;   // units of heads of Q, and of K and of V, that a lane has of an item at most

struct RopeMat {
    uint16_t* p;
    int64_t row, head;               // strides in elements
};

struct RopeParams {
    RopeMat q, k, v, qo, ko, vo;
    int32_t rows, q_heads, kv_heads, d, rot;
    int32_t interleaved, back;
    int32_t units, v_units;          // of a head of Q or K: units of pairs to turn; of a head of V: units to copy
    int32_t q_copies, k_copies;      // units of a head to copy: 0 where the output is the input
    int32_t each, g;                 // lanes of a head: the most units that any has; heads side by side in a warp
    int32_t items;                   // of a row, each with q_each heads of Q and k_each of K and V (the last ones with fewer)
    int32_t q_each, k_each;
    const void* positions;           // int64 or int32, a row each
    int32_t positions64;
    const int64_t* slots;            // rows of ko and vo (else the row itself); one outside [0, slot_rows) is not stored
    int64_t slot_rows;
    float magnitude;
    uint64_t turn[kRopeMaxPairs];    // turns a position of each pair, in 2^-64
};

// W: values of a vector (8, 4, 2 or 1) that divides a head's parts and their places in memory.
cudaError_t launch_rope(const RopeParams& p, int W, int sms, cudaStream_t stream);

}  // namespace lora
